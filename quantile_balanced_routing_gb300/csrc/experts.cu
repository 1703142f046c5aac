// The routed experts of a few tokens (C ABI: moe_mxfp4_experts).  In pieces (pieces.cuh) five kernels: x split by
// route, gate and up, SiTU-GLU split, down, and the tokens' sums; else (mxfp4_stream.cuh) three: gate, up and SiTU-GLU,
// down, sums.  256 tokens' 16 routes over 896 experts, 3584 / 1024: 780 us, 1370 with three kernels.
//
// [K3-width] 延伸解读 on deployment: routed-expert weights in MXFP4; Q&A SiTU-GLU and
// RMSNorm: the experts' activation and the norm of their weighted sum.
#include "mxfp4_stream.cuh"
#include "pieces.cuh"

#include <math.h>

namespace {

// act [R, M] from the slabs' parts [slabs, 2, R, M] of gate and up, for the routes that have an expert.
__global__ void __launch_bounds__(256) k_glu_sum(int slabs, int R, int M, int E, const int32_t* __restrict__ idx,
                                                 const float* __restrict__ parts, float beta1, float beta2,
                                                 float* __restrict__ act) {
    const long long n = (long long)R * M;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
        const int e = idx[i / M];
        if (e < 0 || e >= E) continue;
        float g = 0.0f, u = 0.0f;
        for (int s = 0; s < slabs; ++s) g += parts[2 * s * n + i], u += parts[(2 * s + 1) * n + i];
        act[i] = situ_glu(g, u, beta1, beta2);
    }
}

struct CombineArgs {
    int T, k, E, L, slabs;
    const int32_t* idx;
    const float* w;
    const float* rows;     // [slabs, T k, L]
    const float* gamma;
    float eps;
    __nv_bfloat16* y;
    long long ldy;
};
constexpr int kCombineThreads = 512, kCombineKeep = 2;

// Four elements of a token's weighted sum, its routes in order; the loads of eight routes before the first
// is used.  n routes have an expert: `row` is theirs.
QB_DEV float4 weighted(const CombineArgs& a, const int* row, const float* w, int n, int f) {
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int b = 0; b < a.slabs; ++b) {
        const float* rows = a.rows + (long long)b * a.T * a.k * a.L + f;
        for (int i0 = 0; i0 < n; i0 += 8) {
            float4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i0 + i < n) v[i] = __ldcg(reinterpret_cast<const float4*>(rows + (long long)row[i0 + i] * a.L));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i0 + i >= n) break;
                s.x = fmaf(w[i0 + i], v[i].x, s.x); s.y = fmaf(w[i0 + i], v[i].y, s.y);
                s.z = fmaf(w[i0 + i], v[i].z, s.z); s.w = fmaf(w[i0 + i], v[i].w, s.w);
            }
        }
    }
    return s;
}

// A token a CTA: the weighted sum of its routes, and its norm.  Sums of up to
// kCombineKeep 4 kCombineThreads features stay in registers; wider ones are formed again.
__global__ void __launch_bounds__(kCombineThreads) k_combine(const CombineArgs a) {
    __shared__ float part[kCombineThreads / 32];
    __shared__ int row[QBMOE_MAX_TOPK], routes;
    __shared__ float w[QBMOE_MAX_TOPK];
    const int t = blockIdx.x;
    if (threadIdx.x < 32) {   // the routes that have an expert, in order
        const int r = t * a.k + threadIdx.x, e = (int)threadIdx.x < a.k ? a.idx[r] : -1;
        const unsigned have = __ballot_sync(0xffffffffu, e >= 0 && e < a.E);
        const int at = __popc(have & ((1u << threadIdx.x) - 1));
        if (have >> threadIdx.x & 1) row[at] = r, w[at] = a.w[r];
        if (threadIdx.x == 0) routes = __popc(have);
    }
    __syncthreads();
    pdl_wait();
    const int n = a.L >> 2, m = routes;
    float4 keep[kCombineKeep];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < kCombineKeep; ++i) {
        const int at = threadIdx.x + i * kCombineThreads;
        if (at < n) keep[i] = weighted(a, row, w, m, 4 * at);
    }
    auto square = [&](const float4& v) { ss = fmaf(v.x, v.x, fmaf(v.y, v.y, fmaf(v.z, v.z, fmaf(v.w, v.w, ss)))); };
#pragma unroll
    for (int i = 0; i < kCombineKeep; ++i)
        if ((int)threadIdx.x + i * kCombineThreads < n) square(keep[i]);
    for (int at = threadIdx.x + kCombineKeep * kCombineThreads; at < n; at += kCombineThreads) square(weighted(a, row, w, m, 4 * at));
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
    __syncthreads();
    ss = 0.0f;
    for (int i = 0; i < kCombineThreads / 32; ++i) ss += part[i];
    const float r = __fdiv_rn(1.0f, __fsqrt_rn(ss / (float)a.L + a.eps));
    auto store = [&](int at, const float4& v) {
        const float z[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            a.y[t * a.ldy + 4 * at + j] = __float2bfloat16_rn(a.gamma ? z[j] * r * a.gamma[4 * at + j] : z[j]);
    };
#pragma unroll
    for (int i = 0; i < kCombineKeep; ++i)
        if ((int)threadIdx.x + i * kCombineThreads < n) store(threadIdx.x + i * kCombineThreads, keep[i]);
    for (int at = threadIdx.x + kCombineKeep * kCombineThreads; at < n; at += kCombineThreads) store(at, weighted(a, row, w, m, 4 * at));
}

// Scratch of an experts call: act; gate and up in slabs; the routes' rows.  In pieces: x's pieces where the rows
// come later, gate and up where act would be, act's pieces, and what a split leaves.
struct ExpertsScratch {
    size_t act, parts, rows, act_pieces, offsets, row_map, odd, bytes;
    bool pieces;
    ExpertsScratch(int T, int k, int L, int M) {
        const size_t R = (size_t)T * k, up = slabs_of(L), down = slabs_of(M, kDown);
        pieces = qbh::pieces_ok(L) && qbh::pieces_ok(M) && slabs_of(L) == 1 && slabs_of(M) == 1;
        if (pieces) {
            act = parts = 0;
            rows = qbh::align_up(2 * R * M * 4, 256);
            act_pieces = rows + max(qbh::align_up(down * R * L * 4, 256), qbh::piece_bytes(R, L));
            offsets = act_pieces + qbh::piece_bytes(R, M);
            row_map = offsets + qbh::align_up((QBMOE_MAX_EXPERTS + 1) * 4, 256);
            odd = row_map + qbh::align_up(R * 4, 256);
            bytes = odd + R * qbh::kOddBytes;
            return;
        }
        act = 0;
        parts = qbh::align_up(R * M * 4, 256);
        rows = parts + (up > 1 ? qbh::align_up(up * 2 * R * M * 4, 256) : 0);
        bytes = rows + qbh::align_up(down * R * L * 4, 256);
    }
};

}  // namespace

namespace qbh {

int experts_init() {
    int rc = set_smem_all<QBMOE_BF16, kGlu>();
    if (!rc) rc = set_smem_all<QBMOE_MXFP8, kGlu>();
    if (!rc) rc = set_smem_all<QBMOE_F32, kDown>();
    return rc;
}

}  // namespace qbh

extern "C" size_t qbmoe_mxfp4_experts_workspace_bytes(int T, int k, int L, int M) {
    if (T < 0 || k < 1 || k > QBMOE_MAX_TOPK || (long long)T * k > QBMOE_MAX_ROUTES || !depth_ok(L) || !depth_ok(M)) return 0;
    return ExpertsScratch(T, k, L, M).bytes;
}

extern "C" int moe_mxfp4_experts(int T, int k, int E, int L, int M, int x_type, const void* x, long long ldx,
                                 const uint8_t* x_scales, const int32_t* idx, const float* w,
                                 const uint8_t* gate_codes, const uint8_t* gate_scales, const uint8_t* up_codes,
                                 const uint8_t* up_scales, const uint8_t* out_codes, const uint8_t* out_scales,
                                 float beta1, float beta2, const float* gamma, float rms_eps, void* y, long long ldy,
                                 void* workspace, size_t workspace_bytes, qbmoe_stream_t stream) {
    if (T < 0 || k < 1 || k > QBMOE_MAX_TOPK || (long long)T * k > QBMOE_MAX_ROUTES || E < 1 || E > QBMOE_MAX_EXPERTS ||
        !depth_ok(L) || !depth_ok(M) || !rows_ok(L, x_type, ldx) || ldy < L)
        return QBMOE_EINVAL;
    // (an activation is at most beta1 beta2, so that it is finite or NaN)
    if (!(beta1 > 0.0f) || !(beta2 > 0.0f) || !(beta1 * beta2 <= 0x1p127f) || !(rms_eps >= 0.0f) || !isfinite(rms_eps)) return QBMOE_EINVAL;
    if (T == 0) return QBMOE_OK;
    if (!all_aligned16({x, gate_codes, gate_scales, up_codes, up_scales, out_codes, out_scales}) || !y || !at_bytes(y, 2) ||
        !idx || !at_bytes(idx, 4) || !w || !at_bytes(w, 4) || !at_bytes(gamma, 4) || (x_type == QBMOE_MXFP8 && !all_aligned16({x_scales})))
        return QBMOE_EINVAL;
    if (!workspace || !at_bytes(workspace, 256)) return QBMOE_EINVAL;
    if (workspace_bytes < qbmoe_mxfp4_experts_workspace_bytes(T, k, L, M)) return QBMOE_EWORKSPACE;
    const int rc = qbh::device_init();
    if (rc) return rc;
    const ExpertsScratch at(T, k, L, M);
    char* base = static_cast<char*>(workspace);
    float *act = reinterpret_cast<float*>(base + at.act), *parts = reinterpret_cast<float*>(base + at.parts), *rows = reinterpret_cast<float*>(base + at.rows);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int R = T * k;
    const bool in_pieces = at.pieces && qbh::pieces_pay(min(E, R), R, 3LL * L * M);
    int rc2 = 0;
    if (in_pieces) {
        uint8_t *xp = reinterpret_cast<uint8_t*>(rows), *ap = reinterpret_cast<uint8_t*>(base + at.act_pieces);
        int32_t *offsets = reinterpret_cast<int32_t*>(base + at.offsets), *row_map = reinterpret_cast<int32_t*>(base + at.row_map);
        uint8_t* odd = reinterpret_cast<uint8_t*>(base + at.odd);
        const qbh::PieceSource from{x_type, x, ldx, x_scales, row_map, k, odd};
        if ((rc2 = qbh::split_routes(T, k, E, L, from, idx, xp, offsets, row_map, odd, s))) return rc2;
        if ((rc2 = qbh::piece_product({R, E, M, L, xp, xp + qbh::piece_code_bytes(R, L), gate_codes, gate_scales, up_codes, up_scales,
                                       offsets, nullptr, act, QBMOE_F32, 2LL * M, from, true}, s)))
            return rc2;
        if ((rc2 = qbh::split_glu(R, E, M, act, beta1, beta2, offsets, ap, s))) return rc2;
        if ((rc2 = qbh::piece_product({R, E, L, M, ap, ap + qbh::piece_code_bytes(R, M), out_codes, out_scales, nullptr, nullptr,
                                       offsets, row_map, rows, QBMOE_F32, L, {}, true}, s)))
            return rc2;
    } else {
        StreamArgs a{};
        a.R = R; a.E = E; a.N = M; a.K = L;
        a.x_type = x_type; a.x = x; a.ldx = ldx; a.x_scales = x_scales;
        a.scales = gate_scales; a.scales2 = up_scales;
        a.idx = idx; a.k = k;
        a.y_type = QBMOE_F32; a.y = slabs_of(L) > 1 ? parts : act; a.ldy = M;
        a.beta1 = beta1; a.beta2 = beta2;
        rc2 = x_type == QBMOE_BF16 ? ::stream<QBMOE_BF16, kGlu>(a, gate_codes, up_codes, s) : ::stream<QBMOE_MXFP8, kGlu>(a, gate_codes, up_codes, s);
        if (rc2) return rc2;
        if (slabs_of(L) > 1) {
            const long long blocks = ((long long)R * M + 255) / 256;
            k_glu_sum<<<(unsigned)min(blocks, 8LL * qbh::sm_count()), 256, 0, s>>>(slabs_of(L), R, M, E, idx, parts, beta1, beta2, act);
            if ((rc2 = qbh::cuda_err(cudaGetLastError()))) return rc2;
        }
        a.N = L; a.K = M;
        a.x_type = QBMOE_F32; a.x = act; a.ldx = M; a.x_scales = nullptr;
        a.scales = out_scales; a.scales2 = nullptr;
        a.y = rows; a.ldy = L;
        if ((rc2 = ::stream<QBMOE_F32, kDown>(a, out_codes, nullptr, s))) return rc2;
    }
    const CombineArgs c{T, k, E, L, in_pieces ? 1 : slabs_of(M, kDown), idx, w, rows, gamma, rms_eps, static_cast<__nv_bfloat16*>(y), ldy};
    return qbh::launch_pdl(k_combine, dim3(T), dim3(kCombineThreads), 0, s, c);
}
