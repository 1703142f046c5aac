// MXFP4 tensors (C ABI: moe_mxfp4_*): quantisation of rows, the product of
// MXFP4 rows with MXFP4 weights, and the product's gradients.
//
// [K3-width] 延伸解读 on deployment: routed-expert weights in MXFP4 with
// quantisation-aware post-training.  OCP MX: E2M1 elements, one E8M0 scale per
// 32 along K.
#include "mxfp4.cuh"
#include "mxfp4_decode.cuh"

#include <type_traits>

namespace {

using namespace qb;

// ---------------------------------------------------------------------------
// Quantisation.  Four consecutive lanes hold one block of 32 (8 elements each);
// the block's largest magnitude is two shuffles away.
// ---------------------------------------------------------------------------
constexpr int kQThreads = 256;

// 8 elements of a row from 16-byte loads.
template <typename T> struct Eight;
template <> struct Eight<float> {
    static QB_DEV void load(const float* p, float (&x)[8]) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    static QB_DEV void store(float* p, const float (&x)[8]) {
        reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
};
template <> struct Eight<__nv_bfloat16> {
    static QB_DEV void load(const __nv_bfloat16* p, float (&x)[8]) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
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

// Two floats to a byte of E2M1 codes (lo in the low nibble): round to nearest,
// ties to even, magnitudes above 6 to 6.
QB_DEV uint32_t e2m1_pair(float lo, float hi) {
    uint16_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tmov.b16 %0, {t, 0};\n\t}"
        : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

template <typename T, bool kValues>
__global__ void __launch_bounds__(kQThreads) k_mxfp4_quantize(long long rows, int K, const T* __restrict__ x,
                                                              long long ldx, uint8_t* __restrict__ codes,
                                                              uint8_t* __restrict__ scales, T* __restrict__ values) {
    pdl_trigger();   // a product of these rows may set itself up meanwhile
    const int per_row = K / 8;   // a multiple of 4: the lanes of a block share its fate
    const long long items = rows * per_row;
    for (long long it = (long long)blockIdx.x * kQThreads + threadIdx.x; it < items;
         it += (long long)gridDim.x * kQThreads) {
        const long long r = it / per_row;
        const int k = (int)(it - r * per_row) * 8;
        float v[8];
        Eight<T>::load(x + r * ldx + k, v);
        uint32_t m = 0;   // largest magnitude as bits: an infinity or a NaN is above every finite number
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
        const uint32_t group = 0xfu << (threadIdx.x & 28);
        m = max(m, __shfl_xor_sync(group, m, 1));
        m = max(m, __shfl_xor_sync(group, m, 2));
        // a subnormal maximum has exponent field 0: below 2^-126, so e < -127 and the clamp holds
        const int e = max((int)(m >> 23) - 127 - 2, -127);
        const bool bad = m >= 0x7f800000u;
        const float inv = __int_as_float((127 - e) << 23);   // 2^-e: -127 <= e <= 125 (not used when bad)
        uint32_t q = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) q |= e2m1_pair(v[2 * i] * inv, v[2 * i + 1] * inv) << (8 * i);
        if (bad) q = 0;
        reinterpret_cast<uint32_t*>(codes)[it] = q;
        const uint32_t sb = bad ? 0xffu : (uint32_t)(e + 127);
        if ((threadIdx.x & 3) == 0) scales[it >> 2] = (uint8_t)sb;
        if (kValues) {
            const float sc = e8m0_value(sb);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = e2m1_value(q >> (4 * i)) * sc;
            Eight<T>::store(values + r * K + k, v);
        }
    }
}

bool rows_ok(int K, int x_type, long long ldx) {
    return (x_type == QBMOE_F32 || x_type == QBMOE_BF16) && ldx >= K && ldx % (x_type == QBMOE_BF16 ? 8 : 4) == 0;
}

bool product_sizes_ok(int R, int E, int N, int K, const int32_t* offsets) {
    return R >= 0 && E >= 1 && E <= QBMOE_MAX_EXPERTS && N >= 8 && N % 8 == 0 && K >= 32 && K % 32 == 0 &&
           (offsets || E == 1);
}
int check_workspace(const void* ws, size_t bytes, int R, int E, int N, int K) {
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return QBMOE_EINVAL;
    return bytes < qbmoe_mxfp4_workspace_bytes(R, E, N, K) ? QBMOE_EWORKSPACE : QBMOE_OK;
}
template <typename... P>
bool all_aligned16(const P*... p) { return ((p != nullptr && qbh::aligned16(p)) && ...); }

}  // namespace

namespace qbh {

int mx_quantize(long long rows, int K, int x_type, const void* x, long long ldx, uint8_t* codes, uint8_t* scales,
                void* values, cudaStream_t s) {
    const long long items = rows * (K / 8);
    const int grid = (int)min((items + kQThreads - 1) / kQThreads, 8LL * sm_count());
    auto go = [&](auto tag, auto with) {
        using T = decltype(tag);
        k_mxfp4_quantize<T, decltype(with)::value><<<grid, kQThreads, 0, s>>>(
            rows, K, static_cast<const T*>(x), ldx, codes, scales, static_cast<T*>(values));
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

extern "C" size_t qbmoe_mxfp4_workspace_bytes(int R, int E, int N, int K) {
    if (R < 0 || E < 1 || E > QBMOE_MAX_EXPERTS || N < 8 || N % 8 || K < 32 || K % 32) return 0;
    // codes and scales of rows that come in another type
    return 256 + qbh::align_up((size_t)R * (K / 2), 256) + qbh::align_up((size_t)R * (K / 32), 256);
}

extern "C" int moe_mxfp4_matmul(int R, int E, int N, int K, int x_type, const void* x, long long ldx,
                                const uint8_t* x_scales, const uint8_t* w_codes, const uint8_t* w_scales,
                                const int32_t* offsets, void* y, long long ldy, void* workspace,
                                size_t workspace_bytes, qbmoe_stream_t stream) {
    if (!product_sizes_ok(R, E, N, K, offsets) || ldy < N || ldy % 8) return QBMOE_EINVAL;
    if (x_type == QBMOE_MXFP4 ? ldx != K : !rows_ok(K, x_type, ldx)) return QBMOE_EINVAL;
    int rc = check_workspace(workspace, workspace_bytes, R, E, N, K);
    if (rc) return rc;
    if (R == 0) return QBMOE_OK;
    if (!all_aligned16(static_cast<const uint8_t*>(x), w_codes, w_scales, static_cast<const uint8_t*>(y)) ||
        !qbh::aligned16(offsets) || (x_type == QBMOE_MXFP4 && !all_aligned16(x_scales)))
        return QBMOE_EINVAL;
    if ((rc = qbh::device_init())) return rc;
    uint8_t* codes = static_cast<uint8_t*>(workspace);
    uint8_t* scales = codes + qbh::align_up((size_t)R * (K / 2), 256);
    const bool raw = x_type != QBMOE_MXFP4;
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
                               void* workspace, size_t workspace_bytes, qbmoe_stream_t stream) {
    if (!product_sizes_ok(R, E, N, K, offsets) || lddy < N || lddy % 8 || lddx < K || lddx % 8) return QBMOE_EINVAL;
    int rc = check_workspace(workspace, workspace_bytes, R, E, N, K);
    if (rc) return rc;
    if (R == 0) return QBMOE_OK;
    if (!all_aligned16(static_cast<const uint8_t*>(dy), w_codes, w_scales, static_cast<const uint8_t*>(dx)) ||
        !qbh::aligned16(offsets))
        return QBMOE_EINVAL;
    if ((rc = qbh::device_init())) return rc;
    qbh::MxGrad g{};
    g.weights = false;
    g.R = R; g.E = E; g.N = N; g.K = K;
    g.dy = dy; g.lddy = lddy;
    g.codes = w_codes; g.scales = w_scales; g.offsets = offsets;
    g.out = dx; g.ldo = lddx; g.out_type = QBMOE_BF16;
    return qbh::mx_grad(g, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int moe_mxfp4_wgrad(int R, int E, int N, int K, const void* dy, long long lddy, const uint8_t* x_codes,
                               const uint8_t* x_scales, const int32_t* offsets, int dw_dtype, void* dw,
                               void* workspace, size_t workspace_bytes, qbmoe_stream_t stream) {
    if (!product_sizes_ok(R, E, N, K, offsets) || lddy < N || lddy % 8) return QBMOE_EINVAL;
    if (dw_dtype != QBMOE_F32 && dw_dtype != QBMOE_BF16) return QBMOE_EINVAL;
    int rc = check_workspace(workspace, workspace_bytes, R, E, N, K);
    if (rc) return rc;
    if (!dw || !qbh::aligned16(dw) || !qbh::aligned16(offsets)) return QBMOE_EINVAL;
    if (R > 0 && !all_aligned16(static_cast<const uint8_t*>(dy), x_codes, x_scales)) return QBMOE_EINVAL;
    if ((rc = qbh::device_init())) return rc;
    qbh::MxGrad g{};
    g.weights = true;
    g.R = R; g.E = E; g.N = N; g.K = K;
    g.dy = dy; g.lddy = lddy;
    g.codes = x_codes; g.scales = x_scales; g.offsets = offsets;
    g.out = dw; g.ldo = K; g.out_type = dw_dtype;
    return qbh::mx_grad(g, reinterpret_cast<cudaStream_t>(stream));
}
