// MXFP4 weights with few rows (C ABI: moe_mxfp4_matvec): in pieces where weights are many (pieces.cuh), else with the
// rows in registers (mxfp4_stream.cuh).
//
// [K3-width] 延伸解读 on deployment: MXFP4 weights.
#include "mxfp4_stream.cuh"
#include "pieces.cuh"

namespace {

// y = the slabs' parts [slabs, R, N] added in order, for the rows that an expert owns.
__global__ void __launch_bounds__(256) k_slab_sum(int slabs, int R, int N, int E, const int32_t* __restrict__ offsets,
                                                  const float* __restrict__ parts, int y_type, void* y, long long ldy) {
    const int lo = offsets ? max(offsets[0], 0) : 0, hi = offsets ? min(offsets[E], R) : R;
    const long long n = (long long)max(hi - lo, 0) * N;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
        const long long r = lo + i / N;
        const int f = (int)(i % N);
        float v = 0.0f;
        for (int s = 0; s < slabs; ++s) v += parts[((long long)s * R + r) * N + f];
        if (y_type == QBMOE_F32) static_cast<float*>(y)[r * ldy + f] = v;
        else static_cast<__nv_bfloat16*>(y)[r * ldy + f] = __float2bfloat16_rn(v);
    }
}

// Scratch of a call: parts of the slabs; or the rows' pieces, their offsets and odd bytes.  It is sized without E: pieces
// that pay for as many experts as there are rows have their place, also where a call of fewer experts does without.
constexpr long long kMostPieces = 1LL << 25;   // elements of x that are split: 143 MB of pieces
struct MatvecScratch {
    size_t offsets = 0, odd = 0, bytes = 0;
    bool pieces;
    MatvecScratch(int R, int N, int K) {
        pieces = qbh::pieces_ok(K) && slabs_of(K) == 1 && (long long)R * K <= kMostPieces &&
                 qbh::pieces_pay(min(R, QBMOE_MAX_EXPERTS), R, (long long)N * K);   // for some E
        if (pieces) {
            offsets = qbh::piece_bytes(R, K);
            odd = offsets + qbh::align_up((QBMOE_MAX_EXPERTS + 1) * 4, 256);
            bytes = odd + (size_t)R * qbh::kOddBytes;
        } else if (slabs_of(K) > 1) {
            bytes = (size_t)slabs_of(K) * R * N * 4;
        }
    }
};

}  // namespace

namespace qbh {

int matvec_init() {
    const int rc = set_smem_all<QBMOE_BF16, kStore>();
    return rc ? rc : set_smem_all<QBMOE_MXFP8, kStore>();
}

}  // namespace qbh

extern "C" size_t qbmoe_mxfp4_matvec_workspace_bytes(int R, int N, int K) {
    if (R < 0 || R > QBMOE_MAX_ROWS || N < 8 || N % 8 || N > kMaxCols || !depth_ok(K)) return 0;
    return MatvecScratch(R, N, K).bytes;
}

extern "C" int moe_mxfp4_matvec(int R, int E, int N, int K, int x_type, const void* x, long long ldx,
                                const uint8_t* x_scales, const uint8_t* w_codes, const uint8_t* w_scales,
                                const int32_t* offsets, int y_type, void* y, long long ldy, void* workspace,
                                size_t workspace_bytes, qbmoe_stream_t stream) {
    if (R < 0 || R > QBMOE_MAX_ROWS || E < 1 || E > QBMOE_MAX_EXPERTS || (!offsets && E != 1) || !depth_ok(K) || N < 8 || N % 8 ||
        N > kMaxCols || (long long)E * N > 0x7fffffffLL || !rows_ok(K, x_type, ldx) || ldy < N || (y_type != QBMOE_F32 && y_type != QBMOE_BF16))
        return QBMOE_EINVAL;
    const MatvecScratch at(R, N, K);
    const size_t need = at.bytes;
    if (need && (!workspace || !at_bytes(workspace, 256))) return QBMOE_EINVAL;
    if (workspace_bytes < need) return QBMOE_EWORKSPACE;
    if (R == 0) return QBMOE_OK;
    if (!all_aligned16({x, w_codes, w_scales}) || !y || !at_bytes(y, y_type == QBMOE_F32 ? 4 : 2) || !at_bytes(offsets, 4) ||
        (x_type == QBMOE_MXFP8 && !all_aligned16({x_scales})))
        return QBMOE_EINVAL;
    const int rc = qbh::device_init();
    if (rc) return rc;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (at.pieces && qbh::pieces_pay(min(E, R), R, (long long)N * K)) {
        uint8_t* pieces = static_cast<uint8_t*>(workspace);
        int32_t* piece_offsets = reinterpret_cast<int32_t*>(pieces + at.offsets);
        const qbh::PieceSource from{x_type, x, ldx, x_scales, nullptr, 1, pieces + at.odd};
        const int rc2 = qbh::split_rows(R, E, K, from, offsets, pieces, piece_offsets, pieces + at.odd, s);
        if (rc2) return rc2;
        return qbh::piece_product({R, E, N, K, pieces, pieces + qbh::piece_code_bytes(R, K), w_codes, w_scales, nullptr, nullptr,
                                   offsets ? piece_offsets : nullptr, nullptr, y, y_type, ldy, from, false}, s);
    }
    StreamArgs a{};
    a.R = R; a.E = E; a.N = N; a.K = K;
    a.x_type = x_type; a.x = x; a.ldx = ldx; a.x_scales = x_scales;
    a.scales = w_scales; a.offsets = offsets;
    const bool slabs = slabs_of(K) > 1;
    a.y_type = slabs ? QBMOE_F32 : y_type;
    a.y = slabs ? workspace : y;
    a.ldy = slabs ? N : ldy;
    const int rc2 = x_type == QBMOE_BF16 ? ::stream<QBMOE_BF16, kStore>(a, w_codes, nullptr, s) : ::stream<QBMOE_MXFP8, kStore>(a, w_codes, nullptr, s);
    if (rc2 || !slabs) return rc2;
    const long long blocks = ((long long)R * N + 255) / 256;
    k_slab_sum<<<(unsigned)min(blocks, 8LL * qbh::sm_count()), 256, 0, s>>>(slabs_of(K), R, N, E, offsets, static_cast<float*>(workspace), y_type, y, ldy);
    return qbh::cuda_err(cudaGetLastError());
}
