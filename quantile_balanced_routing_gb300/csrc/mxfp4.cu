// MXFP4 tensors (C ABI: moe_mxfp4_*): quantisation of rows, the product of
// MXFP4 rows with MXFP4 weights, and the product's gradients.
//
// [K3-width] 延伸解读 on deployment: routed-expert weights in MXFP4 with
// quantisation-aware post-training.  OCP MX: E2M1 elements, one E8M0 scale per
// 32 along K.
#include "mxfp4.cuh"
#include "mxfp4_decode.cuh"

#include <cuda_fp16.h>

#include <type_traits>

namespace {

using namespace qb;

// ---------------------------------------------------------------------------
// Quantisation: one pass over the rows, bound by HBM.  Four consecutive lanes
// hold one block of 32 (8 elements each); the block's largest magnitude is two
// shuffles away.  A thread has kQUnroll pieces in flight, a CTA's width apart.
// Contiguous rows are one long row, so that no index is divided (333 us
// instead of 257 with a division and one piece in flight).  57344 x 3584 fp32 with
// values: 252 us, 6.95 TB/s; 262144 x 3584 bf16 to codes: 357 us, 6.7 TB/s.
// ---------------------------------------------------------------------------
constexpr int kQThreads = 256, kQUnroll = 4;

// 8 elements of a row: loads, the largest magnitude as fp32 bits (an infinity or
// a NaN is above every finite number), the values as fp32, and stores.
template <typename T> struct Eight;
template <> struct Eight<float> {
    float4 a, b;
    QB_DEV void load(const float* p) {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    QB_DEV void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    QB_DEV uint32_t amax() const {
        float x[8];
        get(x);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
        return m;
    }
    static QB_DEV void store(float* p, const float (&x)[8]) {
        reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
};
template <> struct Eight<__nv_bfloat16> {
    uint4 u;
    QB_DEV void load(const __nv_bfloat16* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
    QB_DEV void get(float (&x)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    QB_DEV uint32_t amax() const {   // both halves of a word at once
        const uint32_t m = __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu),
                                    __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
        return max(m & 0xffff0000u, m << 16);
    }
    static QB_DEV void store(__nv_bfloat16* p, const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // exact: at most two significant bits
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Eight floats to eight E2M1 codes (element 0 in the low nibble): round to
// nearest, ties to even, magnitudes above 6 to 6.
QB_DEV uint32_t e2m1_codes(const float (&x)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}
// Eight codes to their values.
QB_DEV void e2m1_values(uint32_t q, float (&x)[8]) {
    uint32_t h[4];   // pairs of fp16
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(q));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// Row blockIdx.y, blockIdx.y + gridDim.y, ... of `items` pieces of 8 elements (a
// multiple of 4, so the lanes of a block share its fate).
template <typename T, bool kValues>
__global__ void __launch_bounds__(kQThreads) k_mxfp4_quantize(long long rows, long long items, const T* __restrict__ x,
                                                              long long ldx, uint8_t* __restrict__ codes,
                                                              uint8_t* __restrict__ scales, T* __restrict__ values) {
    pdl_trigger();   // a product of these rows may set itself up meanwhile
    const long long first = (long long)blockIdx.x * (kQThreads * kQUnroll) + threadIdx.x;
    const uint32_t group = 0xfu << (threadIdx.x & 28);
    for (long long r = blockIdx.y; r < rows; r += gridDim.y) {
        Eight<T> in[kQUnroll];
#pragma unroll
        for (int i = 0; i < kQUnroll; ++i)
            if (first + i * kQThreads < items) in[i].load(x + r * ldx + (first + i * kQThreads) * 8);
#pragma unroll
        for (int i = 0; i < kQUnroll; ++i) {
            const long long at = first + i * kQThreads;
            if (at >= items) break;
            uint32_t m = in[i].amax();
            m = max(m, __shfl_xor_sync(group, m, 1));
            m = max(m, __shfl_xor_sync(group, m, 2));
            // a subnormal maximum has exponent field 0: below 2^-126, so e < -127 and the clamp holds
            const int e = max((int)(m >> 23) - 127 - 2, -127);
            const bool bad = m >= 0x7f800000u;
            const float inv = __int_as_float((127 - e) << 23);   // 2^-e: -127 <= e <= 125 (not used when bad)
            float v[8];
            in[i].get(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= inv;
            const uint32_t q = bad ? 0u : e2m1_codes(v);
            const long long out = r * items + at;
            reinterpret_cast<uint32_t*>(codes)[out] = q;
            const uint32_t sb = bad ? 0xffu : (uint32_t)(e + 127);
            if ((threadIdx.x & 3) == 0) scales[out >> 2] = (uint8_t)sb;
            if (kValues) {
                const float sc = e8m0_value(sb);
                e2m1_values(q, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= sc;
                Eight<T>::store(values + out * 8, v);
            }
        }
    }
}

bool rows_ok(int K, int x_type, long long ldx) {
    return (x_type == QBMOE_F32 || x_type == QBMOE_BF16) && ldx >= K && ldx % (x_type == QBMOE_BF16 ? 8 : 4) == 0;
}

// The kernels index up to 16 rows with 32 bits.
constexpr int kMaxK = 1 << 24;
constexpr long long kMaxStride = 1LL << 27;

bool product_sizes_ok(int R, int E, int N, int K, const int32_t* offsets) {
    return R >= 0 && R <= QBMOE_MAX_ROWS && E >= 1 && E <= QBMOE_MAX_EXPERTS && N >= 8 && N % 8 == 0 && N <= kMaxK && K >= 32 &&
           K % 32 == 0 && K <= kMaxK && (long long)E * N <= 0x7fffffffLL && (offsets || E == 1);
}
bool stride_ok(long long ld, int cols) { return ld >= cols && ld % 8 == 0 && ld <= kMaxStride; }
template <typename... P>
bool all_aligned16(const P*... p) { return ((p != nullptr && qbh::aligned16(p)) && ...); }

}  // namespace

namespace qbh {

int mx_quantize(long long rows, int K, int x_type, const void* x, long long ldx, uint8_t* codes, uint8_t* scales,
                void* values, cudaStream_t s) {
    long long n = rows, items = K / 8;
    if (ldx == K) items *= n, n = 1;
    const dim3 grid((unsigned)((items + kQThreads * kQUnroll - 1) / (kQThreads * kQUnroll)),
                    (unsigned)min(n, 65535LL));
    auto go = [&](auto tag, auto with) {
        using T = decltype(tag);
        k_mxfp4_quantize<T, decltype(with)::value><<<grid, kQThreads, 0, s>>>(
            n, items, static_cast<const T*>(x), ldx, codes, scales, static_cast<T*>(values));
    };
    if (x_type == QBMOE_F32) values ? go(float{}, std::true_type{}) : go(float{}, std::false_type{});
    else values ? go(__nv_bfloat16{}, std::true_type{}) : go(__nv_bfloat16{}, std::false_type{});
    return cuda_err(cudaGetLastError());
}

}  // namespace qbh

extern "C" int moe_mxfp4_quantize(long long rows, int K, int x_type, const void* x, long long ldx, uint8_t* codes,
                                  uint8_t* scales, void* values, qbmoe_stream_t stream) {
    if (K < 32 || K % 32 || rows < 0 || rows > (1LL << 40) / K || !rows_ok(K, x_type, ldx)) return QBMOE_EINVAL;
    if (rows == 0) return QBMOE_OK;
    if (!all_aligned16(x, codes) || !scales || !qbh::aligned16(values)) return QBMOE_EINVAL;
    int rc = qbh::device_init();
    if (rc) return rc;
    return qbh::mx_quantize(rows, K, x_type, x, ldx, codes, scales, values, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t qbmoe_mxfp4_workspace_bytes(int R, int K) {
    if (R < 0 || R > QBMOE_MAX_ROWS || K < 32 || K % 32 || K > kMaxK) return 0;
    // codes and scales of rows that come in another type
    return 256 + qbh::align_up((size_t)R * (K / 2), 256) + qbh::align_up((size_t)R * (K / 32), 256);
}

extern "C" int moe_mxfp4_matmul(int R, int E, int N, int K, int x_type, const void* x, long long ldx,
                                const uint8_t* x_scales, const uint8_t* w_codes, const uint8_t* w_scales,
                                const int32_t* offsets, void* y, long long ldy, void* workspace,
                                size_t workspace_bytes, qbmoe_stream_t stream) {
    if (!product_sizes_ok(R, E, N, K, offsets) || !stride_ok(ldy, N)) return QBMOE_EINVAL;
    if (x_type == QBMOE_MXFP4 ? ldx != K : !rows_ok(K, x_type, ldx)) return QBMOE_EINVAL;
    const bool raw = x_type != QBMOE_MXFP4;
    if (raw && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)) return QBMOE_EINVAL;
    if (raw && workspace_bytes < qbmoe_mxfp4_workspace_bytes(R, K)) return QBMOE_EWORKSPACE;
    if (R == 0) return QBMOE_OK;
    if (!all_aligned16(static_cast<const uint8_t*>(x), w_codes, w_scales, static_cast<const uint8_t*>(y)) ||
        !qbh::aligned16(offsets) || (!raw && !all_aligned16(x_scales)))
        return QBMOE_EINVAL;
    const int rc = qbh::device_init();
    if (rc) return rc;
    uint8_t* codes = static_cast<uint8_t*>(workspace);
    uint8_t* scales = codes + qbh::align_up((size_t)R * (K / 2), 256);
    qbh::MxProduct p{};
    p.R = R; p.E = E; p.N = N; p.K = K;
    p.x_codes = raw ? codes : static_cast<uint8_t*>(const_cast<void*>(x));
    p.x_scales = raw ? scales : const_cast<uint8_t*>(x_scales);
    p.w_codes = w_codes; p.w_scales = w_scales; p.offsets = offsets;
    p.y = y; p.ldy = ldy;
    p.raw = raw ? x : nullptr; p.raw_type = x_type; p.raw_ld = ldx;
    return qbh::mx_product(p, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int moe_mxfp4_dgrad(int R, int E, int N, int K, const void* dy, long long lddy, const uint8_t* w_codes,
                               const uint8_t* w_scales, const int32_t* offsets, void* dx, long long lddx,
                               qbmoe_stream_t stream) {
    if (!product_sizes_ok(R, E, N, K, offsets) || !stride_ok(lddy, N) || !stride_ok(lddx, K)) return QBMOE_EINVAL;
    if (R == 0) return QBMOE_OK;
    if (!all_aligned16(static_cast<const uint8_t*>(dy), w_codes, w_scales, static_cast<const uint8_t*>(dx)) ||
        !qbh::aligned16(offsets))
        return QBMOE_EINVAL;
    const int rc = qbh::device_init();
    if (rc) return rc;
    qbh::MxGrad g{};
    g.weights = false;
    g.R = R; g.E = E; g.N = N; g.K = K;
    g.dy = dy; g.lddy = lddy;
    g.codes = w_codes; g.scales = w_scales; g.offsets = offsets;
    g.out = dx; g.ldo = lddx; g.out_type = QBMOE_BF16;
    return qbh::mx_grad(g, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t qbmoe_mxfp4_wgrad_workspace_bytes(int R, int E, int N, int K) {
    if (R < 0 || R > QBMOE_MAX_ROWS || E < 1 || E > QBMOE_MAX_EXPERTS || N < 8 || N % 8 || N > kMaxK || K < 32 || K % 32 || K > kMaxK)
        return 0;
    const int splits = qbh::mx_wgrad_splits(R, E, N, K);
    return splits > 1 ? (size_t)splits * E * N * K * 4 : 0;
}

extern "C" int moe_mxfp4_wgrad(int R, int E, int N, int K, const void* dy, long long lddy, const uint8_t* x_codes,
                               const uint8_t* x_scales, const int32_t* offsets, int dw_dtype, void* dw,
                               void* workspace, size_t workspace_bytes, qbmoe_stream_t stream) {
    if (!product_sizes_ok(R, E, N, K, offsets) || !stride_ok(lddy, N)) return QBMOE_EINVAL;
    if (dw_dtype != QBMOE_F32 && dw_dtype != QBMOE_BF16) return QBMOE_EINVAL;
    if (!dw || !qbh::aligned16(dw) || !qbh::aligned16(offsets)) return QBMOE_EINVAL;
    if (R > 0 && !all_aligned16(static_cast<const uint8_t*>(dy), x_codes, x_scales)) return QBMOE_EINVAL;
    const size_t need = qbmoe_mxfp4_wgrad_workspace_bytes(R, E, N, K);
    if (need && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)) return QBMOE_EINVAL;
    if (workspace_bytes < need) return QBMOE_EWORKSPACE;
    const int rc = qbh::device_init();
    if (rc) return rc;
    qbh::MxGrad g{};
    g.weights = true;
    g.parts = need ? workspace : nullptr;
    g.R = R; g.E = E; g.N = N; g.K = K;
    g.dy = dy; g.lddy = lddy;
    g.codes = x_codes; g.scales = x_scales; g.offsets = offsets;
    g.out = dw; g.ldo = K; g.out_type = dw_dtype;
    return qbh::mx_grad(g, reinterpret_cast<cudaStream_t>(stream));
}
