// MXFP4 weights with few rows, and the routed experts of a few tokens (C ABI:
// moe_mxfp4_matvec, moe_mxfp4_experts).
//
// [K3-width] 延伸解读 on deployment: routed-expert weights in MXFP4; Q&A SiTU-GLU and
// RMSNorm: the experts' activation and the norm of their weighted sum.
#include "mxfp4.cuh"
#include "mxfp4_decode.cuh"

#include <cuda_fp16.h>

#include <initializer_list>

namespace {

using namespace qb;

constexpr int kThreads = 256, kRows = 8;

// Rows of x: bf16, MXFP8 (codes and scales) or fp32.
struct Rows {
    int type;
    const void* x;
    long long ld;
    const uint8_t* scales;
};

template <int kType>
QB_DEV void load_block(const Rows& r, long long row, int blk, int K, float (&v)[32]) {
    if (kType == QBMOE_BF16) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(r.x) + row * r.ld + blk * 32);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 u = p[i];
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) v[8 * i + 2 * j] = __uint_as_float(w[j] << 16), v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    } else if (kType == QBMOE_F32) {
        const float* p = static_cast<const float*>(r.x) + row * r.ld + blk * 32;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = p[i];
    } else {
        const uint8_t* p = static_cast<const uint8_t*>(r.x) + row * r.ld + blk * 32;
        const float sc = e8m0_value(r.scales[row * (K / 32) + blk]);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            uint32_t h;
            const uint16_t q = reinterpret_cast<const uint16_t*>(p)[i];
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(q));
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            v[2 * i] = f.x * sc;
            v[2 * i + 1] = f.y * sc;
        }
    }
}

// Whole warp: dot products of one weight row with n rows of x, in every lane.
template <int kType>
QB_DEV void dot_rows(const Rows& x, const long long (&row)[kRows], int n, int K, const uint8_t* codes, const uint8_t* scales,
                     float (&acc)[kRows]) {
#pragma unroll
    for (int c = 0; c < kRows; ++c) acc[c] = 0.0f;
    for (int blk = threadIdx.x & 31; blk < K / 32; blk += 32) {
        const uint4 u = reinterpret_cast<const uint4*>(codes)[blk];
        const uint32_t q[4] = {u.x, u.y, u.z, u.w};
        const float sc = e8m0_value(scales[blk]);
        float w[32], v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = e2m1_value(q[i >> 3] >> (4 * (i & 7)));
#pragma unroll
        for (int c = 0; c < kRows; ++c) {
            if (c >= n) break;
            load_block<kType>(x, row[c], blk, K, v);
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 32; ++i) s = fmaf(w[i], v[i], s);
            acc[c] = fmaf(s, sc, acc[c]);
        }
    }
#pragma unroll
    for (int c = 0; c < kRows; ++c)
#pragma unroll
        for (int o = 16; o; o >>= 1) acc[c] += __shfl_xor_sync(0xffffffffu, acc[c], o);
}

struct MatvecArgs {
    int R, E, N, K;
    Rows x;
    const uint8_t *codes, *scales;
    const int32_t* offsets;
    int y_type;
    void* y;
    long long ldy;
};

// A weight row a warp, up to kRows rows of one expert a CTA.
template <int kType>
__global__ void __launch_bounds__(kThreads) k_matvec(const MatvecArgs a) {
    __shared__ int seg[QBMOE_MAX_EXPERTS + 1], toff[QBMOE_MAX_EXPERTS + 1], scratch[kThreads / 32];
    load_groups<kRows, kThreads>(Groups{seg, toff}, a.offsets, a.E, a.R, scratch);
    const int f = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (f >= a.N) return;
    for (int chunk = blockIdx.y; chunk < toff[a.E]; chunk += gridDim.y) {
        int g = 0;
        for (int hi = a.E; hi - g > 1;) {
            const int mid = (g + hi) >> 1;
            if (toff[mid] <= chunk) g = mid; else hi = mid;
        }
        const int r0 = seg[g] + (chunk - toff[g]) * kRows, n = min(kRows, seg[g + 1] - r0);
        long long row[kRows];
        for (int c = 0; c < kRows; ++c) row[c] = r0 + c;
        const long long at = (long long)g * a.N + f;
        float acc[kRows];
        dot_rows<kType>(a.x, row, n, a.K, a.codes + at * (a.K / 2), a.scales + at * (a.K / 32), acc);
        if ((threadIdx.x & 31) == 0)
            for (int c = 0; c < n; ++c) {
                const long long o = (r0 + c) * a.ldy + f;
                if (a.y_type == QBMOE_F32) static_cast<float*>(a.y)[o] = acc[c];
                else static_cast<__nv_bfloat16*>(a.y)[o] = __float2bfloat16_rn(acc[c]);
            }
    }
}

struct ExpertsArgs {
    int T, k, E, L, M;
    Rows x;
    const int32_t* idx;
    const float* w;
    const uint8_t *gate, *gate_s, *up, *up_s, *out, *out_s;
    float beta1, beta2;
    const float* gamma;
    float eps;
    __nv_bfloat16* y;
    long long ldy;
    float *act, *rows;   // [T k, M], [T k, L]
};

// act[r][f]: a feature a warp, a route a CTA row.
template <int kType>
__global__ void __launch_bounds__(kThreads) k_gate_up(const ExpertsArgs a) {
    const int f = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), r = blockIdx.y;
    const int e = a.idx[r];
    if (f >= a.M || e < 0 || e >= a.E) return;
    const long long row[kRows] = {r / a.k}, at = (long long)e * a.M + f;
    float g[kRows], u[kRows];
    dot_rows<kType>(a.x, row, 1, a.L, a.gate + at * (a.L / 2), a.gate_s + at * (a.L / 32), g);
    dot_rows<kType>(a.x, row, 1, a.L, a.up + at * (a.L / 2), a.up_s + at * (a.L / 32), u);
    if ((threadIdx.x & 31) == 0) a.act[(long long)r * a.M + f] = situ_glu(g[0], u[0], a.beta1, a.beta2);
}

__global__ void __launch_bounds__(kThreads) k_down(const ExpertsArgs a) {
    const int f = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), r = blockIdx.y;
    const int e = a.idx[r];
    if (f >= a.L || e < 0 || e >= a.E) return;
    const long long row[kRows] = {r}, at = (long long)e * a.L + f;
    float z[kRows];
    dot_rows<QBMOE_F32>(Rows{QBMOE_F32, a.act, a.M, nullptr}, row, 1, a.M, a.out + at * (a.M / 2), a.out_s + at * (a.M / 32), z);
    if ((threadIdx.x & 31) == 0) a.rows[(long long)r * a.L + f] = z[0];
}

// Element f of a token's weighted sum.
QB_DEV float weighted(const ExpertsArgs& a, int t, int f) {
    float s = 0.0f;
    for (int i = 0; i < a.k; ++i) {
        const long long r = (long long)t * a.k + i;
        const int e = a.idx[r];
        if (e >= 0 && e < a.E) s = fmaf(a.w[r], a.rows[r * a.L + f], s);
    }
    return s;
}
// A token a CTA: the weighted sum of its routes, and its norm.
__global__ void __launch_bounds__(kThreads) k_combine(const ExpertsArgs a) {
    __shared__ float part[kThreads / 32];
    const int t = blockIdx.x;
    float ss = 0.0f;
    for (int f = threadIdx.x; f < a.L; f += kThreads) {
        const float s = weighted(a, t, f);
        ss = fmaf(s, s, ss);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
    __syncthreads();
    ss = 0.0f;
    for (int i = 0; i < kThreads / 32; ++i) ss += part[i];
    const float r = __fdiv_rn(1.0f, __fsqrt_rn(ss / (float)a.L + a.eps));
    for (int f = threadIdx.x; f < a.L; f += kThreads) {
        const float z = weighted(a, t, f);
        a.y[t * a.ldy + f] = __float2bfloat16_rn(a.gamma ? z * r * a.gamma[f] : z);
    }
}

constexpr int kMaxCols = 1 << 24;
bool rows_ok(int K, int x_type, long long ldx) {
    return x_type == QBMOE_MXFP8 ? ldx == K : x_type == QBMOE_BF16 && ldx >= K && ldx % 8 == 0;
}
bool depth_ok(int K) { return K >= 32 && K % 32 == 0 && K <= QBMOE_MATVEC_MAX_K; }
bool all_aligned16(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!p || !qbh::aligned16(p)) return false;
    return true;
}
bool at_bytes(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

extern "C" size_t qbmoe_mxfp4_matvec_workspace_bytes(int R, int N, int K) {
    (void)R; (void)N; (void)K;
    return 0;
}

extern "C" int moe_mxfp4_matvec(int R, int E, int N, int K, int x_type, const void* x, long long ldx,
                                const uint8_t* x_scales, const uint8_t* w_codes, const uint8_t* w_scales,
                                const int32_t* offsets, int y_type, void* y, long long ldy, void* workspace,
                                size_t workspace_bytes, qbmoe_stream_t stream) {
    if (R < 0 || R > QBMOE_MAX_ROWS || E < 1 || E > QBMOE_MAX_EXPERTS || (!offsets && E != 1) || !depth_ok(K) || N < 8 || N % 8 ||
        N > kMaxCols || (long long)E * N > 0x7fffffffLL || !rows_ok(K, x_type, ldx) || ldy < N || (y_type != QBMOE_F32 && y_type != QBMOE_BF16))
        return QBMOE_EINVAL;
    const size_t need = qbmoe_mxfp4_matvec_workspace_bytes(R, N, K);
    if (need && (!workspace || !at_bytes(workspace, 256))) return QBMOE_EINVAL;
    if (workspace_bytes < need) return QBMOE_EWORKSPACE;
    if (R == 0) return QBMOE_OK;
    if (!all_aligned16({x, w_codes, w_scales}) || !y || !at_bytes(y, y_type == QBMOE_F32 ? 4 : 2) || !at_bytes(offsets, 4) ||
        (x_type == QBMOE_MXFP8 && !all_aligned16({x_scales})))
        return QBMOE_EINVAL;
    const int rc = qbh::device_init();
    if (rc) return rc;
    const MatvecArgs a{R, E, N, K, Rows{x_type, x, ldx, x_scales}, w_codes, w_scales, offsets, y_type, y, ldy};
    const dim3 grid((N + kThreads / 32 - 1) / (kThreads / 32), (unsigned)min(((long long)R + kRows - 1) / kRows + min(E, R), 65535LL));
    if (x_type == QBMOE_BF16) k_matvec<QBMOE_BF16><<<grid, kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    else k_matvec<QBMOE_MXFP8><<<grid, kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    return qbh::cuda_err(cudaGetLastError());
}

extern "C" size_t qbmoe_mxfp4_experts_workspace_bytes(int T, int k, int L, int M) {
    if (T < 0 || k < 1 || k > QBMOE_MAX_TOPK || (long long)T * k > QBMOE_MAX_ROUTES || !depth_ok(L) || !depth_ok(M)) return 0;
    return qbh::align_up((size_t)T * k * M * 4, 256) + qbh::align_up((size_t)T * k * L * 4, 256);
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
    if (!(beta1 > 0.0f) || !(beta2 > 0.0f) || !(rms_eps >= 0.0f)) return QBMOE_EINVAL;
    if (T == 0) return QBMOE_OK;
    if (!all_aligned16({x, gate_codes, gate_scales, up_codes, up_scales, out_codes, out_scales}) || !y || !at_bytes(y, 2) ||
        !idx || !at_bytes(idx, 4) || !w || !at_bytes(w, 4) || !at_bytes(gamma, 4) || (x_type == QBMOE_MXFP8 && !all_aligned16({x_scales})))
        return QBMOE_EINVAL;
    if (!workspace || !at_bytes(workspace, 256)) return QBMOE_EINVAL;
    if (workspace_bytes < qbmoe_mxfp4_experts_workspace_bytes(T, k, L, M)) return QBMOE_EWORKSPACE;
    const int rc = qbh::device_init();
    if (rc) return rc;
    float* act = static_cast<float*>(workspace);
    float* rows = reinterpret_cast<float*>(static_cast<char*>(workspace) + qbh::align_up((size_t)T * k * M * 4, 256));
    const ExpertsArgs a{T, k, E, L, M, Rows{x_type, x, ldx, x_scales}, idx, w, gate_codes, gate_scales, up_codes, up_scales, out_codes,
                        out_scales, beta1, beta2, gamma, rms_eps, static_cast<__nv_bfloat16*>(y), ldy, act, rows};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const dim3 up((M + kThreads / 32 - 1) / (kThreads / 32), T * k), down((L + kThreads / 32 - 1) / (kThreads / 32), T * k);
    if (x_type == QBMOE_BF16) k_gate_up<QBMOE_BF16><<<up, kThreads, 0, s>>>(a);
    else k_gate_up<QBMOE_MXFP8><<<up, kThreads, 0, s>>>(a);
    k_down<<<down, kThreads, 0, s>>>(a);
    k_combine<<<T, kThreads, 0, s>>>(a);
    return qbh::cuda_err(cudaGetLastError());
}
