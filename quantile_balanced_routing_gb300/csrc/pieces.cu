// Rows as sums of MXFP4 rows: what goes before a product with few rows and much weight.
#include "pieces.cuh"
#include "mxfp4_stream.cuh"

namespace {

constexpr int kSplitThreads = 256;

// This lane's 8 elements of a block, as the four lanes of the block's quad have them, times 2^up.
struct Block {
    float f[8];
    uint32_t most;  // bits of the largest magnitude of this lane's
    int up;         // exponent of the block's own scale
    bool nan;       // whose scale is NaN
};
QB_DEV uint32_t largest(const float (&f)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7fffffffu);
    return m;
}
template <int kX>
QB_DEV Block block_of(const void* x, long long ldx, const uint8_t* x_scales, int K, long long row, int at) {
    Block b;
    b.up = 0;
    b.nan = false;
    if (kX == QBMOE_MXFP8) {
        const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(x) + row * ldx + 8 * at);
        uint32_t h[4];
        asm("{\n\t.reg .b16 p, q, r, s;\n\tmov.b32 {p, q}, %4;\n\tmov.b32 {r, s}, %5;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, p;\n\tcvt.rn.f16x2.e4m3x2 %1, q;\n\t"
            "cvt.rn.f16x2.e4m3x2 %2, r;\n\tcvt.rn.f16x2.e4m3x2 %3, s;\n\t}"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
            : "r"(q.x), "r"(q.y));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
            b.f[2 * j] = v.x;
            b.f[2 * j + 1] = v.y;
        }
        b.most = largest(b.f);
        const int s = x_scales[row * (K >> 5) + (at >> 2)];
        b.nan = s == 255;
        b.up = s - 127;
    } else {
        const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(x) + row * ldx + 8 * at);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            b.f[2 * j] = __uint_as_float(w[j] << 16), b.f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            m = __vmaxu2(m, w[j] & 0x7fff7fffu);
        }
        b.most = max(m << 16, m & 0xffff0000u);
    }
    return b;
}

// A lane's share of the eight pieces of a block: the codes of its elements, four bytes a piece, and (in lane l
// < 8) the scales of the warp's eight blocks in piece l.
struct Pieces {
    uint32_t codes[qbh::kPieces];
    uint2 scales;
};
// Whole warp.  special: the block has no such pieces (a NaN has: a scale of NaN).
QB_DEV Pieces pieces_of(const Block& b, bool& special) {
    Pieces p;
    uint32_t m = b.most;
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    int e = max((int)(m >> 23) - 127, -100);                 // the largest is in [2^e, 2^(e + 1)), or tiny
    if (m == 0) e = 0;
    bool bad = b.nan || m >= 0x7f800000u;
    int base = 106 + e + (m == 0 ? 0 : b.up);                // piece 0's scale byte: 2^(e - 21)
    special |= m == 0x7f800000u || (m != 0 && m < (27u << 23)) || (!bad && (base < 0 || base + 3 * (qbh::kPieces - 1) > 254));
    if (base < 0 || base + 3 * (qbh::kPieces - 1) > 254) bad = true;
    const float unit = __int_as_float((127 + 21 - e) << 23); // 2^(21 - e)
    // Digits from 0 to 7, 4 too many each: 4 (8^8 - 1) / 7 added to the whole number, which the sum with 1.5 2^23 has
    // in its low bits.  An element's octal digits move to nibbles of their own, the byte selection turns four at
    // once into codes (0xE, 0xD, 0xC, 0xA for -4 .. -1, then 0, 2, 4, 5), two elements' codes share bytes, and those of
    // four pairs change places with the pieces.
    uint32_t pair[4][2];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t u = __float_as_uint(fmaf(bad ? 0.0f : b.f[j], unit, 12582912.0f)) - 0x4b400000u + 9586980u;
        u += (u & 0xfff000u) * 15u;
        u += (u & 0x0fc00fc0u) * 3u;
        u += u & 0x38383838u;
        const uint32_t lo = j & 1 ? 0xa0c0d0e0u : 0x0a0c0d0eu, hi = j & 1 ? 0x50402000u : 0x05040200u;
        const uint32_t a = __byte_perm(lo, hi, u), c = __byte_perm(lo, hi, u >> 16);
        pair[j >> 1][0] = j & 1 ? pair[j >> 1][0] | a : a;
        pair[j >> 1][1] = j & 1 ? pair[j >> 1][1] | c : c;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t a = __byte_perm(pair[0][h], pair[1][h], 0x5140), c = __byte_perm(pair[2][h], pair[3][h], 0x5140);
        const uint32_t d = __byte_perm(pair[0][h], pair[1][h], 0x7362), f = __byte_perm(pair[2][h], pair[3][h], 0x7362);
        p.codes[4 * h] = __byte_perm(a, c, 0x5410);
        p.codes[4 * h + 1] = __byte_perm(a, c, 0x7632);
        p.codes[4 * h + 2] = __byte_perm(d, f, 0x5410);
        p.codes[4 * h + 3] = __byte_perm(d, f, 0x7632);
    }
    const int lane = threadIdx.x & 31;
    const uint32_t byte = (lane & 3) ? 0u : (uint32_t)(bad ? 255 : base) << (8 * (lane >> 2 & 3));
    const uint32_t lo = __reduce_or_sync(0xffffffffu, lane < 16 ? byte : 0u), hi = __reduce_or_sync(0xffffffffu, lane < 16 ? 0u : byte);
    p.scales = make_uint2(__vaddus4(lo, 0x03030303u * (lane & 7)), __vaddus4(hi, 0x03030303u * (lane & 7)));   // (NaN stays)
    return p;
}
// Pieces of elements 8 at .. of row `row`; scales lie behind all rows' codes.
QB_DEV void store_pieces(const Pieces& p, uint8_t* codes, uint8_t* scales, long long row, int K, int at) {
    uint8_t* c = codes + row * qbh::kPieces * (K >> 1) + 4 * at;
#pragma unroll
    for (int i = 0; i < qbh::kPieces; ++i) *reinterpret_cast<uint32_t*>(c + (long long)i * (K >> 1)) = p.codes[i];
    const int lane = threadIdx.x & 31;
    if (lane < qbh::kPieces) *reinterpret_cast<uint2*>(scales + (row * qbh::kPieces + lane) * (K >> 5) + (at >> 5) * 8) = p.scales;
}

struct SplitArgs {
    int R, E, K, k;
    const void* x;
    long long ldx;
    const uint8_t* x_scales;
    const int32_t* offsets;     // split_rows
    const int32_t* idx;         // split_routes
    uint8_t *codes, *scales;
    int32_t *piece_offsets, *row_map;
    uint8_t* odd;
};
// Whole warp: the odd byte of its 256 elements; the first's warp clears what is behind the row's last.
QB_DEV void store_odd(uint8_t* odd, long long row, int chunk, int chunks, bool any) {
    const int lane = threadIdx.x & 31;
    if (lane == chunk || (chunk == 0 && lane >= chunks)) odd[row * qbh::kOddBytes + lane] = lane == chunk && any;
}

// A warp 256 elements of a row.
template <int kX>
__global__ void __launch_bounds__(kSplitThreads) k_split_rows(const SplitArgs a) {
    pdl_trigger();
    const int lo = a.offsets ? min(max(a.offsets[0], 0), a.R) : 0, hi = a.offsets ? min(max(a.offsets[a.E], 0), a.R) : a.R;
    if (a.offsets)
        for (int e = blockIdx.x * kSplitThreads + threadIdx.x; e <= a.E; e += gridDim.x * kSplitThreads)
            a.piece_offsets[e] = min(max(a.offsets[e], 0), a.R) * qbh::kPieces;
    const uint32_t lane = threadIdx.x & 31, warps = a.K >> 8, n = max(hi - lo, 0) * warps;   // (at most 2^17)
    for (uint32_t i = blockIdx.x * (kSplitThreads / 32) + (threadIdx.x >> 5); i < n; i += gridDim.x * (kSplitThreads / 32)) {
        const long long row = lo + i / warps;
        const int chunk = i % warps, at = chunk * 32 + lane;
        bool special = false;
        store_pieces(pieces_of(block_of<kX>(a.x, a.ldx, a.x_scales, a.K, row, at), special), a.codes, a.scales, row, a.K, at);
        store_odd(a.odd, row, chunk, warps, __any_sync(0xffffffffu, special));
    }
}

// The same for tokens: a token's pieces go to each of its routes' places in expert order.
template <int kX>
__global__ void __launch_bounds__(kThreads) k_split_routes(const SplitArgs a) {
    extern __shared__ __align__(128) char sm[];
    __shared__ int scratch[kThreads / 32];
    pdl_trigger();
    int* seg = reinterpret_cast<int*>(sm);
    int* first = seg + a.E + 1;
    int* hist = first + a.E + 1;
    uint16_t* list = reinterpret_cast<uint16_t*>(hist + 8 * a.E);
    uint16_t* place = list + a.R;
    StreamArgs g{};
    g.R = a.R;
    g.E = a.E;
    g.idx = a.idx;
    for (int r = threadIdx.x; r < a.R; r += kThreads) place[r] = 0xffff;
    group_rows<kGlu>(g, seg, first, list, hist, scratch);
    const int routes = seg[a.E];
    for (int i = threadIdx.x; i < routes; i += kThreads) place[list[i]] = (uint16_t)i;
    if (blockIdx.x == 0) {
        for (int e = threadIdx.x; e <= a.E; e += kThreads) a.piece_offsets[e] = seg[e] * qbh::kPieces;
        for (int i = threadIdx.x; i < routes; i += kThreads) a.row_map[i] = list[i];
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, warps = a.K >> 8, T = a.R / a.k;
    for (int i = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < T * warps; i += gridDim.x * (kThreads / 32)) {
        const int t = i / warps, chunk = i % warps, at = chunk * 32 + lane;
        bool special = false;
        const Pieces p = pieces_of(block_of<kX>(a.x, a.ldx, a.x_scales, a.K, t, at), special);
        special = __any_sync(0xffffffffu, special);
        for (int j = 0; j < a.k; ++j) {
            const int to = place[t * a.k + j];
            if (to == 0xffff) continue;
            store_pieces(p, a.codes, a.scales, to, a.K, at);
            store_odd(a.odd, to, chunk, warps, special);
        }
    }
}

struct GluArgs {
    int R, E, M;
    const float* h;
    float beta1, beta2;
    const int32_t* piece_offsets;
    uint8_t *codes, *scales;
};
__global__ void __launch_bounds__(kSplitThreads) k_split_glu(const GluArgs a) {
    pdl_trigger();
    pdl_wait();   // h comes from the kernel before
    const uint32_t rows = min(__ldcg(a.piece_offsets + a.E) / qbh::kPieces, a.R), lane = threadIdx.x & 31, warps = a.M >> 8;
    for (uint32_t i = blockIdx.x * (kSplitThreads / 32) + (threadIdx.x >> 5); i < rows * warps; i += gridDim.x * (kSplitThreads / 32)) {
        const long long row = i / warps;
        const int at = (int)(i % warps) * 32 + lane;
        const float4* g = reinterpret_cast<const float4*>(a.h + row * 2 * a.M) + 2 * at;
        const float4* u = g + (a.M >> 2);
        const float4 g0 = __ldcg(g), g1 = __ldcg(g + 1), u0 = __ldcg(u), u1 = __ldcg(u + 1);
        Block b;
        b.up = 0;
        b.nan = false;
        b.f[0] = situ_glu(g0.x, u0.x, a.beta1, a.beta2); b.f[1] = situ_glu(g0.y, u0.y, a.beta1, a.beta2);
        b.f[2] = situ_glu(g0.z, u0.z, a.beta1, a.beta2); b.f[3] = situ_glu(g0.w, u0.w, a.beta1, a.beta2);
        b.f[4] = situ_glu(g1.x, u1.x, a.beta1, a.beta2); b.f[5] = situ_glu(g1.y, u1.y, a.beta1, a.beta2);
        b.f[6] = situ_glu(g1.z, u1.z, a.beta1, a.beta2); b.f[7] = situ_glu(g1.w, u1.w, a.beta1, a.beta2);
        b.most = largest(b.f);
        bool special = false;   // finite, and what is below 2^-121 is as good as zero
        store_pieces(pieces_of(b, special), a.codes, a.scales, row, a.M, at);
    }
}

constexpr int kRoutesSmem = (2 * (QBMOE_MAX_EXPERTS + 1) + 8 * QBMOE_MAX_EXPERTS) * 4 + 2 * QBMOE_MAX_ROUTES * 2;

int grid_of(long long warps_total, int warps_cta, int per_sm) {
    const long long ctas = (warps_total + warps_cta - 1) / warps_cta, most = (long long)per_sm * qbh::sm_count();
    return (int)max(1LL, min(ctas, most));
}

}  // namespace

namespace qbh {

int split_rows(int R, int E, int K, const PieceSource& x, const int32_t* offsets, uint8_t* pieces, int32_t* piece_offsets,
               uint8_t* odd, cudaStream_t s) {
    const SplitArgs a{R, E, K, 1, x.x, x.ldx, x.x_scales, offsets, nullptr, pieces, pieces + piece_code_bytes(R, K), piece_offsets, nullptr, odd};
    const int grid = grid_of((long long)R * (K / 256), kSplitThreads / 32, 6);
    if (x.x_type == QBMOE_MXFP8) k_split_rows<QBMOE_MXFP8><<<grid, kSplitThreads, 0, s>>>(a);
    else k_split_rows<QBMOE_BF16><<<grid, kSplitThreads, 0, s>>>(a);
    return cuda_err(cudaGetLastError());
}

int split_routes(int T, int k, int E, int K, const PieceSource& x, const int32_t* idx, uint8_t* pieces, int32_t* piece_offsets,
                 int32_t* row_map, uint8_t* odd, cudaStream_t s) {
    const SplitArgs a{T * k, E, K, k, x.x, x.ldx, x.x_scales, nullptr, idx, pieces, pieces + piece_code_bytes((long long)T * k, K), piece_offsets, row_map, odd};
    const int grid = grid_of((long long)T * (K / 256), kThreads / 32, 2);
    if (x.x_type == QBMOE_MXFP8) k_split_routes<QBMOE_MXFP8><<<grid, kThreads, kRoutesSmem, s>>>(a);
    else k_split_routes<QBMOE_BF16><<<grid, kThreads, kRoutesSmem, s>>>(a);
    return cuda_err(cudaGetLastError());
}

int split_glu(int R, int E, int M, const float* h, float beta1, float beta2, const int32_t* piece_offsets, uint8_t* pieces, cudaStream_t s) {
    const GluArgs a{R, E, M, h, beta1, beta2, piece_offsets, pieces, pieces + piece_code_bytes(R, M)};
    return launch_pdl(k_split_glu, dim3(grid_of((long long)R * (M / 256), kSplitThreads / 32, 6)), dim3(kSplitThreads), 0, s, a);
}

int pieces_init() {
    const int rc = cuda_err(cudaFuncSetAttribute(k_split_routes<QBMOE_BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRoutesSmem));
    return rc ? rc : cuda_err(cudaFuncSetAttribute(k_split_routes<QBMOE_MXFP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRoutesSmem));
}

}  // namespace qbh
