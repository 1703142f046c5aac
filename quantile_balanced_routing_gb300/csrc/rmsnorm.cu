// The norm in front of a layer (C ABI: moe_add_rmsnorm, moe_add_rmsnorm_backward):
// the residual's addition, the RMS norm of the sum as rows of the input's type or
// in MXFP8, and the gradients.
//
// A row is held in registers between its sum of squares and its outputs, so that each
// input is read once and each output written once.  A thread's pieces are 8
// elements (consecutive where rows are vectors), kNormItems of them a block's width apart; four neighbouring threads
// hold a block of 32, whose largest magnitude is two shuffles away.
//
// Many rows go through k_add_rmsnorm_rows and k_add_rmsnorm_backward_rows: persistent CTAs whose
// next rows come to shared memory by asynchronous copies meanwhile, so that HBM does not wait for a row's
// reduction.  Few rows, short rows and rows off 16-byte boundaries go through the kernels without a ring.
//
// Measured, 16384 x 7168 bf16 with residual: forward to MXFP8 and its values 173 us (6.1 TB/s, 90% of the copy rate; 238
// without the ring), backward with dtotal 161 us (5.8 TB/s; 331, and 189 with the gain read from global memory).
// HBM bounds both.  Rows of odd widths are read an element at a time and bound by issue: 16384 x 2021 bf16, 141 and
// 177 us for a floor of 39.
#include "mxfp4.cuh"

#include <cuda_fp16.h>

#include <math.h>
#include <type_traits>

namespace {

using namespace qb;

constexpr int kNormItems = 4;            // pieces of 8 elements a thread holds
constexpr int kNormThreads = 512;        // most threads of a row
constexpr int kRowWarps = 8;             // rows of a CTA when a warp holds a row
constexpr int kGainParts = 608;          // most partial sums of the gain's gradient (twice as many CTAs of 64 threads:
                                         // 16384 x 2021 bf16, 177 us, 315 with 608)
constexpr int kRingParts = 1520;         // with rows in a ring
constexpr int kRingRow = 512;            // shortest row of a ring

// How a piece of 8 elements lies in its row: together, read at once or one by one; or 32 elements apart, a warp's
// pieces sharing 256 elements, so that the reads of a row off 16-byte boundaries are contiguous over the lanes
// (16384 x 2021 bf16: 141 us, 176 one by one; 4096 x 7001 fp32 88).
enum { kOnes, kVector, kSpread };
template <int kForm>
QB_DEV int element(int i, int j) { return kForm == kSpread ? ((i & ~31) << 3) + 32 * j + (i & 31) : 8 * i + j; }
template <int kForm>
QB_DEV int pieces(int H) { return kForm == kSpread ? (H + 255) >> 8 << 5 : (H + 7) >> 3; }
// Piece i of a row, zeros past its end.
template <typename T, int kForm>
QB_DEV void load8(const T* __restrict__ row, int i, int H, float (&v)[8]) {
    if (kForm == kVector && sizeof(T) == 4) {
        const float4 a = reinterpret_cast<const float4*>(row)[2 * i], b = reinterpret_cast<const float4*>(row)[2 * i + 1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else if (kForm == kVector) {
        const uint4 u = reinterpret_cast<const uint4*>(row)[i];
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) v[2 * j] = __uint_as_float(w[j] << 16), v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = element<kForm>(i, j) < H ? to_f32<T>(row[element<kForm>(i, j)]) : 0.0f;
    }
}
template <typename T, int kForm>
QB_DEV void store8(T* __restrict__ row, int i, int H, const float (&v)[8]) {
    if (kForm == kVector && sizeof(T) == 4) {
        reinterpret_cast<float4*>(row)[2 * i] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(row)[2 * i + 1] = make_float4(v[4], v[5], v[6], v[7]);
    } else if (kForm == kVector) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        reinterpret_cast<uint4*>(row)[i] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (element<kForm>(i, j) < H) row[element<kForm>(i, j)] = from_f32<T>(v[j]);
    }
}

// Sums of kSums values over the threads of a row, the same bits in each: a warp's by
// shuffles, then the warps' sums by shuffles.
template <int kSums>
QB_DEV void row_sum(float (&s)[kSums], float* scratch /* [kSums][kNormThreads / 32] */) {
#pragma unroll
    for (int q = 0; q < kSums; ++q)
#pragma unroll
        for (int o = 16; o; o >>= 1) s[q] += __shfl_xor_sync(0xffffffffu, s[q], o);
    if (blockDim.x == 32) return;
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
    __syncthreads();   // the scratch may still be read for the row before
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int q = 0; q < kSums; ++q) scratch[q * (kNormThreads / 32) + warp] = s[q];
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kSums; ++q) {
        const int lane = threadIdx.x & 31;
        s[q] = lane < warps ? scratch[q * (kNormThreads / 32) + lane] : 0.0f;
#pragma unroll
        for (int o = 16; o; o >>= 1) s[q] += __shfl_xor_sync(0xffffffffu, s[q], o);
    }
}

// The mean square, and 1 / sqrt of it, correctly rounded operations: once a row.
QB_DEV float mean_square(float squares, int H, float eps) { return __fadd_rn(__fdiv_rn(squares, (float)H), eps); }
QB_DEV float inverse_sqrt(float mean) { return __fdiv_rn(1.0f, __fsqrt_rn(mean)); }

// Rows whose sum of squares left fp32's range or came near its least numbers take it again of elements times a
// power of two, so that it lies between 2^-118 and 2^126.  The whole row decides alike, by the sum itself.  (The question
// costs ordinary rows 1 to 4%: 16384 x 7168 bf16 173.2 us for 172.4 without it, the gradient 160.3 for 157.5, 131072 x 512
// 116.2 for 114.7 and 121.0 for 116.1.)
struct Range {
    float least, most;
    QB_DEV bool holds(float squares) const { return squares >= least && squares <= most; }
};
constexpr float kLargest = 0x1.fffffep127f, kSmallMean = 0x1p-80f, kLargeMean = 0x1p60f;
// most: of the mean square with eps.
Range range_of(int H, float eps, float most) {
    return {eps < kSmallMean ? kSmallMean * H : 0.0f, !(eps <= 0.5f * most) ? -1.0f : most < kLargest / 2 / H ? 0.5f * most * H : 0.5f * kLargest};
}
// 1 / rms as a product of two factors, in the order in which neither product leaves the range before its end.
struct Factors {
    float first, second;
};
template <typename F>
QB_DEV Factors rescaled(float mean, int H, float eps, float* scratch, F squares) {
    const float s = mean < kSmallMean ? 0x1p90f : mean <= kLargeMean ? 1.0f : 0x1p-72f;
    float q[1] = {squares(s)};
    row_sum<1>(q, scratch);
    const float r = inverse_sqrt(mean_square(q[0], H, eps * s * s));
    return s > 1.0f ? Factors{s, r} : Factors{r, s};
}
// v times its 1 / rms.
template <int kItems>
QB_DEV void normalise(float (&v)[kItems][8], int items, float mean, int H, float eps, float* scratch) {
    const Factors f = rescaled(mean, H, eps, scratch, [&](float s) {
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            if (threadIdx.x + i * blockDim.x >= items) break;
#pragma unroll
            for (int j = 0; j < 8; ++j) q = fmaf(v[i][j] * s, v[i][j] * s, q);
        }
        return q;
    });
#pragma unroll
    for (int i = 0; i < kItems; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (threadIdx.x + i * blockDim.x < items) v[i][j] = v[i][j] * f.first * f.second;
}

struct NormArgs {
    int T, H;
    const void* x;
    long long ldx;
    const void* residual;
    long long ldr;
    const float* gamma;
    float eps;
    void* total;
    long long ldt;
    void* y;
    long long ldy;
    uint8_t *codes, *scales;
    Range range;
};

// MXFP8 of a block whose 8 elements this thread holds; four neighbouring threads hold it.
QB_DEV void mxfp8_store(float (&n)[8], uint8_t* codes, uint8_t* scale, float (&values)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(n[j]) & 0x7fffffffu);
    const uint32_t group = 0xfu << (threadIdx.x & 28);
    m = max(m, __shfl_xor_sync(group, m, 1));
    m = max(m, __shfl_xor_sync(group, m, 2));
    const int e = max((int)(m >> 23) - 127 - 7, -127);   // an exponent field of 0 is below -127
    const bool bad = m >= 0x7f800000u;
    const float inv = __int_as_float((127 - e) << 23);   // 2^-e: -127 <= e <= 120 (not used when bad)
    uint32_t q[2];
    asm("{\n\t.reg .b16 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 a, %3, %2;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 b, %5, %4;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 c, %7, %6;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 d, %9, %8;\n\t"
        "mov.b32 %0, {a, b};\n\tmov.b32 %1, {c, d};\n\t}"
        : "=r"(q[0]), "=r"(q[1])
        : "f"(n[0] * inv), "f"(n[1] * inv), "f"(n[2] * inv), "f"(n[3] * inv), "f"(n[4] * inv), "f"(n[5] * inv),
          "f"(n[6] * inv), "f"(n[7] * inv));
    if (bad) q[0] = q[1] = 0;
    *reinterpret_cast<uint2*>(codes) = make_uint2(q[0], q[1]);
    if ((threadIdx.x & 3) == 0) *scale = (uint8_t)(bad ? 255 : e + 127);
    const float sc = bad ? __int_as_float(0x7fffffff) : __int_as_float(e > -127 ? (e + 127) << 23 : 0x00400000);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;
        asm("{\n\t.reg .b16 lo, hi, p;\n\tmov.b32 {lo, hi}, %1;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
            : "=r"(h)
            : "r"(q[i >> 1] >> (16 * (i & 1))));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        values[2 * i] = f.x * sc;
        values[2 * i + 1] = f.y * sc;
    }
}

// One row a CTA of blockDim.x threads, or, with blockDim.x = 32, one a warp.
template <typename TX, typename TR, int kForm, bool kQuant>
__global__ void __launch_bounds__(kNormThreads) k_add_rmsnorm(const NormArgs a) {
    __shared__ float scratch[kNormThreads / 32];
    const long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= a.T) return;   // whole warps, and only where a warp holds a row
    const int items = pieces<kForm>(a.H);
    const TX* x = static_cast<const TX*>(a.x) + t * a.ldx;
    float v[kNormItems][8];
#pragma unroll
    for (int i = 0; i < kNormItems; ++i) {
        const int at = threadIdx.x + i * blockDim.x;
        if (at < items) load8<TX, kForm>(x, at, a.H, v[i]);
    }
    if (a.residual) {
        const TR* residual = static_cast<const TR*>(a.residual) + t * a.ldr;
        TR* total = static_cast<TR*>(a.total) + t * a.ldt;
        float r[kNormItems][8];
#pragma unroll
        for (int i = 0; i < kNormItems; ++i) {
            const int at = threadIdx.x + i * blockDim.x;
            if (at < items) load8<TR, kForm>(residual, at, a.H, r[i]);
        }
#pragma unroll
        for (int i = 0; i < kNormItems; ++i) {
            const int at = threadIdx.x + i * blockDim.x;
            if (at >= items) break;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = to_f32<TR>(from_f32<TR>(v[i][j] + r[i][j]));
            store8<TR, kForm>(total, at, a.H, v[i]);
        }
    }
    float ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < kNormItems; ++i) {
        if (threadIdx.x + i * blockDim.x >= items) break;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss[0] = fmaf(v[i][j], v[i][j], ss[0]);
    }
    row_sum<1>(ss, scratch);
    float r = inverse_sqrt(mean_square(ss[0], a.H, a.eps));
    if (!a.range.holds(ss[0])) {
        normalise<kNormItems>(v, items, mean_square(ss[0], a.H, a.eps), a.H, a.eps, scratch);
        r = 1.0f;
    }
#pragma unroll
    for (int i = 0; i < kNormItems; ++i) {
        const int at = threadIdx.x + i * blockDim.x;
        if (at >= items) break;
        float g[8], out[8];
        load8<float, kForm>(a.gamma, at, a.H, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * r * g[j];
        if (kQuant) {
            const long long block = t * (items >> 2) + (at >> 2);
            mxfp8_store(v[i], a.codes + t * a.H + 8 * at, a.scales + block, out);
            if (a.y) store8<__nv_bfloat16, kForm>(static_cast<__nv_bfloat16*>(a.y) + t * a.ldy, at, a.H, out);
        } else {
            store8<TX, kForm>(static_cast<TX*>(a.y) + t * a.ldy, at, a.H, v[i]);
        }
    }
}

// Rows blockIdx.x, + gridDim.x, .. in a ring of `stages` rows of `bytes`.  A thread copies the pieces
// that it reads itself, so the ring needs no barrier: a thread waits for its own copies alone.
struct Ring {
    int stages, bytes;
};
constexpr int kRingStages = 4;

QB_DEV void copy16(char* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
QB_DEV void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest `rows` rows of this thread's copies have landed.
QB_DEV void copies_wait(int rows) {
    if (rows == 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (rows == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (rows == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}
// The gain in shared memory, the two halves of each piece apart: 16 bytes a thread without conflicts.
QB_DEV void gain_to_smem(float4* g, const float* gamma, int items) {
    for (int i = threadIdx.x; i < 2 * items; i += blockDim.x) g[(i & 1) * items + (i >> 1)] = reinterpret_cast<const float4*>(gamma)[i];
}
QB_DEV void gain8(const float4* gain, int at, int items, float (&g)[8]) {
    const float4 a = gain[at], b = gain[items + at];
    g[0] = a.x; g[1] = a.y; g[2] = a.z; g[3] = a.w; g[4] = b.x; g[5] = b.y; g[6] = b.z; g[7] = b.w;
}
// This thread's pieces of 8 elements of a row.
template <typename T, int kItems>
QB_DEV void copy_row(char* dst, const T* row, int items) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int at = threadIdx.x + i * blockDim.x;
        if (at >= items) break;
#pragma unroll
        for (int b = 0; b < 8 * (int)sizeof(T); b += 16)
            copy16(dst + 8 * at * (int)sizeof(T) + b, reinterpret_cast<const char*>(row + 8 * at) + b);
    }
}

template <typename TX, typename TR, bool kQuant, int kItems>
__global__ void __launch_bounds__(kNormThreads, kItems == 2 ? 2 : 1) k_add_rmsnorm_rows(const NormArgs a, const Ring ring) {
    extern __shared__ __align__(128) char sm[];
    __shared__ float scratch[kNormThreads / 32];
    const int items = a.H >> 3, x_bytes = a.H * (int)sizeof(TX);
    long long next = blockIdx.x;
    auto bring = [&](int s) {
        if (next < a.T) {
            char* dst = sm + s * ring.bytes;
            copy_row<TX, kItems>(dst, static_cast<const TX*>(a.x) + next * a.ldx, items);
            if (a.residual) copy_row<TR, kItems>(dst + x_bytes, static_cast<const TR*>(a.residual) + next * a.ldr, items);
        }
        next += gridDim.x;
        copies_commit();
    };
    for (int i = 0; i < ring.stages; ++i) bring(i);
    int s = 0;
    for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
        copies_wait(ring.stages - 1);
        const TX* x = reinterpret_cast<const TX*>(sm + s * ring.bytes);
        const TR* residual = reinterpret_cast<const TR*>(sm + s * ring.bytes + x_bytes);
        float v[kItems][8], ss[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int at = threadIdx.x + i * blockDim.x;
            if (at >= items) break;
            load8<TX, kVector>(x, at, a.H, v[i]);
            if (a.residual) {
                float r[8];
                load8<TR, kVector>(residual, at, a.H, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = to_f32<TR>(from_f32<TR>(v[i][j] + r[j]));
                store8<TR, kVector>(static_cast<TR*>(a.total) + t * a.ldt, at, a.H, v[i]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) ss[0] = fmaf(v[i][j], v[i][j], ss[0]);
        }
        bring(s);   // this thread has read its pieces
        if (++s == ring.stages) s = 0;
        row_sum<1>(ss, scratch);
        float r = inverse_sqrt(mean_square(ss[0], a.H, a.eps));
        if (!a.range.holds(ss[0])) {
            normalise<kItems>(v, items, mean_square(ss[0], a.H, a.eps), a.H, a.eps, scratch);
            r = 1.0f;
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int at = threadIdx.x + i * blockDim.x;
            if (at >= items) break;
            float g[8], out[8];
            load8<float, kVector>(a.gamma, at, a.H, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * r * g[j];
            if (kQuant) {
                mxfp8_store(v[i], a.codes + t * a.H + 8 * at, a.scales + t * (items >> 2) + (at >> 2), out);
                if (a.y) store8<__nv_bfloat16, kVector>(static_cast<__nv_bfloat16*>(a.y) + t * a.ldy, at, a.H, out);
            } else {
                store8<TX, kVector>(static_cast<TX*>(a.y) + t * a.ldy, at, a.H, v[i]);
            }
        }
    }
}

// Of a row's gradient out of range: 1 / rms as two factors, and the mean of g times the normed row.  `squares` and
// `products` are the row's sums over this thread's pieces.
struct GradFactors {
    Factors f;
    float whole, rest;   // 1 / rms itself, and 1, unless it passes the range
    float mean;
};
template <typename F, typename P>
QB_DEV GradFactors grad_rescaled(float mean, int H, float eps, float* scratch, F squares, P products) {
    GradFactors g;
    g.f = rescaled(mean, H, eps, scratch, squares);
    float q[1] = {products(g.f)};
    row_sum<1>(q, scratch);
    g.mean = q[0] / (float)H;
    const float whole = g.f.first * g.f.second;
    g.whole = whole <= kLargest ? whole : g.f.first;
    g.rest = whole <= kLargest ? 1.0f : g.f.second;
    return g;
}
struct NormGradArgs {
    int T, H;
    const void* dn;
    long long lddn;
    const void* total;
    long long ldt;
    const float* gamma;
    float eps;
    const void* dtotal;
    long long lddt;
    void* dx;
    long long lddx;
    float* parts;   // [gridDim.x, H] sums of dn total r, or NULL
    Range range;
    // Whether a row's gradient is formed of the sums at hand: the products' must be finite, too.
    QB_DEV bool ordinary(const float (&s)[2]) const { return range.holds(s[0]) && fabsf(s[1]) <= kLargest; }
};

// Rows blockIdx.x * blockDim.y + threadIdx.y, + gridDim.x * blockDim.y, ...: the sums of
// squares and of g total are taken together; the gain's gradient adds up in registers.
template <typename TD, typename TT, int kForm>
__global__ void __launch_bounds__(kNormThreads) k_add_rmsnorm_backward(const NormGradArgs a) {
    __shared__ float scratch[2 * (kNormThreads / 32)];
    extern __shared__ float lines[];   // [blockDim.y][H] where a warp holds a row
    const int items = pieces<kForm>(a.H);
    float acc[kNormItems][8] = {};
    for (long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y; t < a.T; t += (long long)gridDim.x * blockDim.y) {
        float d[kNormItems][8], v[kNormItems][8], s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kNormItems; ++i) {
            const int at = threadIdx.x + i * blockDim.x;
            if (at >= items) break;
            load8<TD, kForm>(static_cast<const TD*>(a.dn) + t * a.lddn, at, a.H, d[i]);
            load8<TT, kForm>(static_cast<const TT*>(a.total) + t * a.ldt, at, a.H, v[i]);
        }
#pragma unroll
        for (int i = 0; i < kNormItems; ++i) {
            const int at = threadIdx.x + i * blockDim.x;
            if (at >= items) break;
            float g[8];
            load8<float, kForm>(a.gamma, at, a.H, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] = fmaf(v[i][j], v[i][j], s[0]), s[1] = fmaf(d[i][j] * g[j], v[i][j], s[1]);
        }
        row_sum<2>(s, scratch);
        if (!a.ordinary(s)) {
            // (the row is read again, so that the ordinary row's registers are its own)
            const TD* dn = static_cast<const TD*>(a.dn) + t * a.lddn;
            const TT* total = static_cast<const TT*>(a.total) + t * a.ldt;
            const GradFactors f = grad_rescaled(mean_square(s[0], a.H, a.eps), a.H, a.eps, scratch, [&](float scale) {
                float q = 0.0f;
                for (int at = threadIdx.x; at < items; at += blockDim.x) {
                    float x[8];
                    load8<TT, kForm>(total, at, a.H, x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) q = fmaf(x[j] * scale, x[j] * scale, q);
                }
                return q;
            }, [&](const Factors& f) {
                float q = 0.0f;
                for (int at = threadIdx.x; at < items; at += blockDim.x) {
                    float y[8], x[8], g[8];
                    load8<TD, kForm>(dn, at, a.H, y);
                    load8<TT, kForm>(total, at, a.H, x);
                    load8<float, kForm>(a.gamma, at, a.H, g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) q = fmaf(y[j] * g[j], x[j] * f.first * f.second, q);
                }
                return q;
            });
#pragma unroll
            for (int i = 0; i < kNormItems; ++i) {
                const int at = threadIdx.x + i * blockDim.x;
                if (at >= items) break;
                float y[8], x[8], g[8], o[8] = {};
                load8<TD, kForm>(dn, at, a.H, y);
                load8<TT, kForm>(total, at, a.H, x);
                load8<float, kForm>(a.gamma, at, a.H, g);
                if (a.dtotal) load8<TT, kForm>(static_cast<const TT*>(a.dtotal) + t * a.lddt, at, a.H, o);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float n = x[j] * f.f.first * f.f.second;
                    acc[i][j] = fmaf(y[j], n, acc[i][j]);
                    o[j] += (y[j] * g[j] - n * f.mean) * f.whole * f.rest;
                }
                store8<TT, kForm>(static_cast<TT*>(a.dx) + t * a.lddx, at, a.H, o);
            }
            continue;
        }
        const float r = inverse_sqrt(mean_square(s[0], a.H, a.eps)), c = s[1] / (float)a.H * r * r;
#pragma unroll
        for (int i = 0; i < kNormItems; ++i) {
            const int at = threadIdx.x + i * blockDim.x;
            if (at >= items) break;
            float g[8], o[8] = {};
            load8<float, kForm>(a.gamma, at, a.H, g);
            if (a.dtotal) load8<TT, kForm>(static_cast<const TT*>(a.dtotal) + t * a.lddt, at, a.H, o);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                acc[i][j] = fmaf(d[i][j], v[i][j] * r, acc[i][j]);
                o[j] += (d[i][j] * g[j] - v[i][j] * c) * r;
            }
            store8<TT, kForm>(static_cast<TT*>(a.dx) + t * a.lddx, at, a.H, o);
        }
    }
    if (!a.parts) return;
    float* part = a.parts + (long long)blockIdx.x * a.H;
    if (blockDim.y == 1) {
#pragma unroll
        for (int i = 0; i < kNormItems; ++i) {
            const int at = threadIdx.x + i * blockDim.x;
            if (at < items) store8<float, kForm == kSpread ? kSpread : kOnes>(part, at, a.H, acc[i]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kNormItems; ++i) {
        const int at = threadIdx.x + i * blockDim.x;
        if (at < items) store8<float, kForm == kSpread ? kSpread : kOnes>(lines + threadIdx.y * a.H, at, a.H, acc[i]);
    }
    __syncthreads();
    for (int j = threadIdx.y * 32 + threadIdx.x; j < a.H; j += 32 * kRowWarps) {
        float s = 0.0f;
        for (int w = 0; w < kRowWarps; ++w) s += lines[w * a.H + j];
        part[j] = s;
    }
}

// The same over a ring of rows: dn, total and dtotal are read twice from shared memory, which leaves
// registers for the gain's sums.
template <typename TD, typename TT, int kItems>
__global__ void __launch_bounds__(kNormThreads, kItems == 2 ? 2 : 1) k_add_rmsnorm_backward_rows(const NormGradArgs a, const Ring ring) {
    extern __shared__ __align__(128) char smem[];
    __shared__ float scratch[2 * (kNormThreads / 32)];
    const int items = a.H >> 3, d_bytes = a.H * (int)sizeof(TD), t_bytes = a.H * (int)sizeof(TT);
    float4* gain = reinterpret_cast<float4*>(smem);
    char* sm = smem + a.H * 4;
    long long next = blockIdx.x;
    auto bring = [&](int s) {
        if (next < a.T) {
            char* dst = sm + s * ring.bytes;
            copy_row<TD, kItems>(dst, static_cast<const TD*>(a.dn) + next * a.lddn, items);
            copy_row<TT, kItems>(dst + d_bytes, static_cast<const TT*>(a.total) + next * a.ldt, items);
            if (a.dtotal) copy_row<TT, kItems>(dst + d_bytes + t_bytes, static_cast<const TT*>(a.dtotal) + next * a.lddt, items);
        }
        next += gridDim.x;
        copies_commit();
    };
    for (int i = 0; i < ring.stages; ++i) bring(i);
    gain_to_smem(gain, a.gamma, items);
    __syncthreads();
    float acc[kItems][8] = {};
    int s = 0;
    for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
        copies_wait(ring.stages - 1);
        const TD* dn = reinterpret_cast<const TD*>(sm + s * ring.bytes);
        const TT* total = reinterpret_cast<const TT*>(sm + s * ring.bytes + d_bytes);
        const TT* dtotal = reinterpret_cast<const TT*>(sm + s * ring.bytes + d_bytes + t_bytes);
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int at = threadIdx.x + i * blockDim.x;
            if (at >= items) break;
            float d[8], v[8], g[8];
            load8<TD, kVector>(dn, at, a.H, d);
            load8<TT, kVector>(total, at, a.H, v);
            gain8(gain, at, items, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[0] = fmaf(v[j], v[j], sum[0]), sum[1] = fmaf(d[j] * g[j], v[j], sum[1]);
        }
        row_sum<2>(sum, scratch);
        if (a.ordinary(sum)) {
            const float r = inverse_sqrt(mean_square(sum[0], a.H, a.eps)), c = sum[1] / (float)a.H * r * r;
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                const int at = threadIdx.x + i * blockDim.x;
                if (at >= items) break;
                float d[8], v[8], g[8], o[8] = {};
                load8<TD, kVector>(dn, at, a.H, d);
                load8<TT, kVector>(total, at, a.H, v);
                gain8(gain, at, items, g);
                if (a.dtotal) load8<TT, kVector>(dtotal, at, a.H, o);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    acc[i][j] = fmaf(d[j], v[j] * r, acc[i][j]);
                    o[j] += (d[j] * g[j] - v[j] * c) * r;
                }
                store8<TT, kVector>(static_cast<TT*>(a.dx) + t * a.lddx, at, a.H, o);
            }
        } else {
            const GradFactors f = grad_rescaled(mean_square(sum[0], a.H, a.eps), a.H, a.eps, scratch, [&](float scale) {
                float q = 0.0f;
                for (int at = threadIdx.x; at < items; at += blockDim.x) {
                    float v[8];
                    load8<TT, kVector>(total, at, a.H, v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) q = fmaf(v[j] * scale, v[j] * scale, q);
                }
                return q;
            }, [&](const Factors& f) {
                float q = 0.0f;
                for (int at = threadIdx.x; at < items; at += blockDim.x) {
                    float d[8], v[8], g[8];
                    load8<TD, kVector>(dn, at, a.H, d);
                    load8<TT, kVector>(total, at, a.H, v);
                    gain8(gain, at, items, g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) q = fmaf(d[j] * g[j], v[j] * f.first * f.second, q);
                }
                return q;
            });
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                const int at = threadIdx.x + i * blockDim.x;
                if (at >= items) break;
                float d[8], v[8], g[8], o[8] = {};
                load8<TD, kVector>(dn, at, a.H, d);
                load8<TT, kVector>(total, at, a.H, v);
                gain8(gain, at, items, g);
                if (a.dtotal) load8<TT, kVector>(dtotal, at, a.H, o);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float n = v[j] * f.f.first * f.f.second;
                    acc[i][j] = fmaf(d[j], n, acc[i][j]);
                    o[j] += (d[j] * g[j] - n * f.mean) * f.whole * f.rest;
                }
                store8<TT, kVector>(static_cast<TT*>(a.dx) + t * a.lddx, at, a.H, o);
            }
        }
        bring(s);   // this thread has read its pieces
        if (++s == ring.stages) s = 0;
    }
    if (!a.parts) return;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int at = threadIdx.x + i * blockDim.x;
        if (at < items) store8<float, kVector>(a.parts + (long long)blockIdx.x * a.H, at, a.H, acc[i]);
    }
}

// dgamma: the parts of 32 columns a CTA, kFinishRows runs of them added in order.
constexpr int kFinishRows = 32;
__global__ void __launch_bounds__(32 * kFinishRows) k_gain_finish(int parts, int H, const float* __restrict__ part,
                                                     float* __restrict__ dgamma) {
    __shared__ float line[kFinishRows][33];
    const int j = blockIdx.x * 32 + threadIdx.x;
    float s = 0.0f;
    if (j < H) {
#pragma unroll 8
        for (int p = threadIdx.y; p < parts; p += kFinishRows) s += part[(long long)p * H + j];
    }
    line[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && j < H) {
        for (int w = 1; w < kFinishRows; ++w) s += line[w][threadIdx.x];
        dgamma[j] = s;
    }
}

bool float_type(int t) { return t == QBMOE_F32 || t == QBMOE_BF16; }
int size_of(int t) { return t == QBMOE_F32 ? 4 : 2; }
bool at_elements(const void* p, int type) { return (reinterpret_cast<uintptr_t>(p) & (size_of(type) - 1)) == 0; }
// Rows that are read in 16-byte pieces.
bool vectors(const void* p, long long ld, int type) { return qbh::aligned16(p) && ld * size_of(type) % 16 == 0; }
bool sizes_ok(int T, int H, float eps) {
    return T >= 0 && T <= QBMOE_MAX_ROWS && H >= 1 && H <= QBMOE_MAX_NORM && eps >= 0.0f && isfinite(eps);
}
// A warp a row up to 1024 elements, else the threads that hold a row in kNormItems pieces each.
dim3 row_block(int H) {
    const int threads = ((H + 8 * kNormItems - 1) / (8 * kNormItems) + 31) & ~31;
    return threads <= 32 ? dim3(32, kRowWarps) : dim3(threads);
}
int gain_parts(int T, int H) {
    const long long ctas = (T + (long long)row_block(H).y - 1) / row_block(H).y;
    const long long most = row_block(H).y == 1 && row_block(H).x <= 64 ? 2 * kGainParts : kGainParts;   // eight small CTAs a SM
    return (int)(ctas < most ? ctas : most);
}

// Whether the rows go through a ring, and its shape: up to rows of 8192 as many CTAs a SM as 64 registers a thread
// and `least` rows (and the gain, where it is read twice a row) each in shared memory allow, one beyond.  Measured in us with
// a ring and without, forward and (with dtotal) backward, bf16, GPU time (floor: bytes at the copy rate):
//   310 x 7168 (3)       8, 7     13, 21       65536 x 2048 (158)  178, 201   183, 322
//   1000 x 7168 (8)     12, 12    19, 32       65536 x 1056 (81)   100, 137   138, 228
//   8192 x 7168 (69)    79, 109   87, 177      65536 x 1024 (79)    92, 108    99, 165
//   8192 x 3584 (35)    42, 55    53, 91       131072 x 512 (79)   116, 123   121, 178
// Forward, a ring is no better for fp32 alone (8192 x 4096: 88, 83), whose 16-byte reads meet in shared memory's banks,
// nor with two rows (fp32, 8192 x 7168: 154, 143).  What the rule leaves: 200000 x 256 (61: 100, 125; 133, 156), and fp32's
// gradient (8192 x 4096: 97, 106).
constexpr int kRingBytes = 224 * 1024;     // a SM's
constexpr int kRingCta = 112 * 1024;
constexpr int kWide = 8192;
struct RingShape {
    Ring ring;
    bool use;
    int grid, threads;
    size_t smem;
};
RingShape ring_of(int T, int H, int bytes, int gain_bytes, int least, bool able) {
    const int items = H > kWide ? 4 : 2;
    RingShape r{};
    r.threads = ((H + 8 * items - 1) / (8 * items) + 31) & ~31;
    int per_sm = H > kWide ? 1 : max(2, 1024 / r.threads);
    r.ring.bytes = bytes;
    for (;; --per_sm) {
        r.ring.stages = (kRingBytes / per_sm - (per_sm > 2 ? 1280 : 0) - gain_bytes) / bytes;   // (a CTA's own KB, and its sums)
        if (r.ring.stages >= least || per_sm <= 2) break;
    }
    if (r.ring.stages > kRingStages) r.ring.stages = kRingStages;
    r.grid = per_sm * qbh::sm_count();
    if (r.grid > kRingParts) r.grid = kRingParts;
    r.smem = gain_bytes + (size_t)r.ring.stages * bytes;
    r.use = able && H >= kRingRow && T >= r.grid && r.ring.stages >= least;
    return r;
}

// Calls f with a value of each of two types.
template <typename F>
void with_types(int first, int second, F f) {
    if (first == QBMOE_F32) second == QBMOE_F32 ? f(float{}, float{}) : f(float{}, __nv_bfloat16{});
    else second == QBMOE_F32 ? f(__nv_bfloat16{}, float{}) : f(__nv_bfloat16{}, __nv_bfloat16{});
}

template <typename K>
int allow_ring(K kern, int bytes) {
    return qbh::cuda_err(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
}

}  // namespace

namespace qbh {

int rmsnorm_init() {
    int rc = 0;
    for (int i = 0; i < 4 && !rc; ++i)
        with_types(i & 1 ? QBMOE_BF16 : QBMOE_F32, i & 2 ? QBMOE_BF16 : QBMOE_F32, [&](auto first, auto second) {
            using A = decltype(first);
            using B = decltype(second);
            rc = allow_ring(k_add_rmsnorm_rows<A, B, false, 2>, kRingCta);
            if (!rc) rc = allow_ring(k_add_rmsnorm_rows<A, B, true, 2>, kRingCta);
            if (!rc) rc = allow_ring(k_add_rmsnorm_rows<A, B, false, 4>, kRingBytes);
            if (!rc) rc = allow_ring(k_add_rmsnorm_rows<A, B, true, 4>, kRingBytes);
            if (!rc) rc = allow_ring(k_add_rmsnorm_backward_rows<A, B, 2>, kRingCta);
            if (!rc) rc = allow_ring(k_add_rmsnorm_backward_rows<A, B, 4>, kRingBytes);
        });
    return rc;
}

}  // namespace qbh

extern "C" int moe_add_rmsnorm(int T, int H, int x_type, const void* x, long long ldx, int res_type,
                               const void* residual, long long ldr, const float* gamma, float eps, void* total,
                               long long ldt, void* y, long long ldy, uint8_t* codes, uint8_t* scales,
                               qbmoe_stream_t stream) {
    if (!sizes_ok(T, H, eps) || !float_type(x_type) || (codes && H % 32) || !codes != !scales) return QBMOE_EINVAL;
    if (ldx < H || (y && ldy < H) || !residual != !total) return QBMOE_EINVAL;
    if (residual && (!float_type(res_type) || ldr < H || ldt < H)) return QBMOE_EINVAL;
    if (T == 0) return QBMOE_OK;
    const int y_type = codes ? QBMOE_BF16 : x_type;
    if (!x || !gamma || (!y && !codes) || !at_elements(x, x_type) || !at_elements(gamma, QBMOE_F32) || !at_elements(y, y_type) ||
        (reinterpret_cast<uintptr_t>(codes) & 7u))
        return QBMOE_EINVAL;
    if (residual && (!at_elements(residual, res_type) || !at_elements(total, res_type))) return QBMOE_EINVAL;
    const int rc = qbh::device_init();
    if (rc) return rc;
    const bool vec = H % 8 == 0 && vectors(x, ldx, x_type) && vectors(gamma, 0, QBMOE_F32) && vectors(y, y ? ldy : 0, y_type) &&
                     (!residual || (vectors(residual, ldr, res_type) && vectors(total, ldt, res_type)));
    const NormArgs a{T, H, x, ldx, residual, ldr, gamma, eps, total, ldt, y, ldy, codes, scales, range_of(H, eps, kLargest)};
    const dim3 block = row_block(H);
    const unsigned grid = (unsigned)(((long long)T + block.y - 1) / block.y);
    const RingShape rows = ring_of(T, H, H * (size_of(x_type) + (residual ? size_of(res_type) : 0)), 0, 3, vec && (x_type == QBMOE_BF16 || (residual && res_type == QBMOE_BF16)));
    with_types(x_type, residual ? res_type : x_type, [&](auto tx, auto tr) {
        using TX = decltype(tx);
        using TR = decltype(tr);
        if (rows.use) {
            auto stream_rows = [&](auto kern) {
                kern<<<rows.grid, rows.threads, rows.smem, reinterpret_cast<cudaStream_t>(stream)>>>(a, rows.ring);
            };
            if (H <= kWide) codes ? stream_rows(k_add_rmsnorm_rows<TX, TR, true, 2>) : stream_rows(k_add_rmsnorm_rows<TX, TR, false, 2>);
            else codes ? stream_rows(k_add_rmsnorm_rows<TX, TR, true, 4>) : stream_rows(k_add_rmsnorm_rows<TX, TR, false, 4>);
            return;
        }
        auto go = [&](auto kern) { kern<<<grid, block, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a); };
        if (vec) codes ? go(k_add_rmsnorm<TX, TR, kVector, true>) : go(k_add_rmsnorm<TX, TR, kVector, false>);
        else codes ? go(k_add_rmsnorm<TX, TR, kOnes, true>) : go(k_add_rmsnorm<TX, TR, kSpread, false>);   // (a block of codes is four threads')
    });
    return qbh::cuda_err(cudaGetLastError());
}

extern "C" size_t qbmoe_add_rmsnorm_workspace_bytes(int T, int H) {
    return sizes_ok(T, H, 0.0f) ? (size_t)min(T, kRingParts) * H * 4 : 0;   // (gain_parts, or a ring's grid, at most)
}

extern "C" int moe_add_rmsnorm_backward(int T, int H, int dn_type, const void* dn, long long lddn, int total_type,
                                        const void* total, long long ldt, const float* gamma, float eps,
                                        const void* dtotal, long long lddt, void* dx, long long lddx, float* dgamma,
                                        void* workspace, size_t workspace_bytes, qbmoe_stream_t stream) {
    if (!sizes_ok(T, H, eps) || !float_type(dn_type) || !float_type(total_type)) return QBMOE_EINVAL;
    if (lddn < H || ldt < H || lddx < H || (dtotal && lddt < H) || !at_elements(dgamma, QBMOE_F32)) return QBMOE_EINVAL;
    if (T > 0 && (!dn || !total || !gamma || !dx || !at_elements(dn, dn_type) || !at_elements(total, total_type) ||
                  !at_elements(gamma, QBMOE_F32) || !at_elements(dtotal, total_type) || !at_elements(dx, total_type)))
        return QBMOE_EINVAL;
    if (T > 0 && dgamma) {
        if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return QBMOE_EINVAL;
        if (workspace_bytes < qbmoe_add_rmsnorm_workspace_bytes(T, H)) return QBMOE_EWORKSPACE;
    }
    if (T == 0 && !dgamma) return QBMOE_OK;
    const int rc = qbh::device_init();
    if (rc) return rc;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) return qbh::cuda_err(cudaMemsetAsync(dgamma, 0, (size_t)H * 4, s));
    const bool vec = H % 8 == 0 && vectors(dn, lddn, dn_type) && vectors(total, ldt, total_type) &&
                     vectors(gamma, 0, QBMOE_F32) && vectors(dtotal, dtotal ? lddt : 0, total_type) &&
                     vectors(dx, lddx, total_type);
    float* parts = dgamma ? static_cast<float*>(workspace) : nullptr;
    const NormGradArgs a{T, H, dn, lddn, total, ldt, gamma, eps, dtotal, lddt, dx, lddx, parts, range_of(H, eps, kLargeMean)};
    const dim3 block = row_block(H);
    const RingShape rows = ring_of(T, H, H * (size_of(dn_type) + size_of(total_type) * (dtotal ? 2 : 1)), H * 4, 2, vec && (dn_type == QBMOE_BF16 || total_type == QBMOE_BF16));
    const int grid = rows.use ? rows.grid : gain_parts(T, H);
    const size_t smem = block.y > 1 ? (size_t)kRowWarps * H * 4 : 0;
    with_types(dn_type, total_type, [&](auto td, auto tt) {
        using TD = decltype(td);
        using TT = decltype(tt);
        if (rows.use) {
            if (H <= kWide) k_add_rmsnorm_backward_rows<TD, TT, 2><<<grid, rows.threads, rows.smem, s>>>(a, rows.ring);
            else k_add_rmsnorm_backward_rows<TD, TT, 4><<<grid, rows.threads, rows.smem, s>>>(a, rows.ring);
            return;
        }
        if (vec) k_add_rmsnorm_backward<TD, TT, kVector><<<grid, block, smem, s>>>(a);
        else k_add_rmsnorm_backward<TD, TT, kSpread><<<grid, block, smem, s>>>(a);
    });
    if (dgamma) k_gain_finish<<<(H + 31) / 32, dim3(32, kFinishRows), 0, s>>>(grid, H, parts, dgamma);
    return qbh::cuda_err(cudaGetLastError());
}
