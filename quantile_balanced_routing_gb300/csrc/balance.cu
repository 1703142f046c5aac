// Router training (C ABI: moe_balance_loss, moe_router_backward): the balance
// loss of a routed batch with its per-expert counts, and the gradient of the
// router logits from the mixture weights and from that loss.
//
// Notation: s = sigmoid(x), c = 1 - s, S_t = sum_j s_tj, p_tj = s_tj / S_t.
// Both kernels make one pass over the [T, n] logits with one warp per token:
// a lane keeps n / 32 of the row in registers, so S_t (and, in the backward
// pass, sum_j f_j s_tj) is a warp reduction and no row is read twice.
#include "common.cuh"

namespace {

using namespace qb;

constexpr int kBalWarps = 8;
constexpr int kBalThreads = 32 * kBalWarps;
constexpr int kMaxPerLane = QBMOE_MAX_EXPERTS / 32;   // 32 logits of a row per lane
constexpr float kLogitLimit = 80.0f;

// e = exp(-x) and s = 1 / (1 + e) = sigmoid(x), x clamped to [-80, 80] and a NaN kept.
// exp(-x) = 2^t (1 + r + ..) for the rounded t = -x log2 e, with r = -x - t ln 2: the
// rounding of t alone would put up to 4e-6 into e, and r is below 2^-17.  With the
// hardware exponential (2^-22) and reciprocal (2^-23) s is within 2^-21 of its value at
// every x (measured: shares of a token within 3.2e-7, which is fp32's own rounding).
// Forming the bits of the router's own, exactly specified score instead takes 17 us
// more (loss 40 against 23, gradient 44 against 26, 16384 x 896 fp32) for shares within
// 2.6e-7; uncorrected, loss 19 and gradient 24 for 3.8e-6.
QB_DEV float score(float x, float& e) {
    float c;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(x), "f"(-kLogitLimit));
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(c) : "f"(kLogitLimit));
    const float t = c * -1.4426950408889634f;
    float r = fmaf(t, -0.693147182464599609375f, -c);   // ln 2 as a float, and the rest of it
    r = fmaf(t, 1.9046543e-9f, r);
    float u;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(u) : "f"(t));   // no subnormal between the limits
    e = fmaf(u, r, u);
    float s;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
    return s;
}
// s and its derivative s (1 - s) = m - m^2 for the smaller m of s and 1 - s = e s: the
// relative error is that of m (e s^2 would have that of s twice), also where s rounds
// to 1.  0 where the clamp holds.
QB_DEV float score_slope(float x, float& slope) {
    float e;
    const float s = score(x, e);
    const float m = fminf(s, e * s);
    slope = fabsf(x) > kLogitLimit ? 0.0f : fmaf(-m, m, m);
    return s;
}

template <typename T> struct Vec;   // elements of T in 16 bytes
template <> struct Vec<float> { static constexpr int n = 4; };
template <> struct Vec<__nv_bfloat16> { static constexpr int n = 8; };

// This lane's elements of a row: element v of group i is column (32 i + lane) V + v.
template <typename T, int V>
QB_DEV void load_row(const T* __restrict__ row, int n, int lane, float (&x)[kMaxPerLane]) {
#pragma unroll
    for (int i = 0; i < kMaxPerLane / V; ++i) {
        const int j = (32 * i + lane) * V;
        if (V == 1) {
            x[i] = j < n ? to_f32<T>(row[j]) : 0.0f;
        } else if (j < n) {   // n is a multiple of V here
            const uint4 u = *reinterpret_cast<const uint4*>(row + j);
            const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
            for (int v = 0; v < V; ++v) x[i * V + v] = to_f32<T>(e[v]);
        }
    }
}

QB_DEV float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Largest q with off[q] <= t (off[0] <= t assumed).
QB_DEV int find_seq(const int32_t* off, int S, int t) {
    int lo = 0, hi = S;
    while (hi - lo > 1) {
        const int mid = lo + ((hi - lo) >> 1);
        if (__ldg(off + mid) <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// ---------------------------------------------------------------------------
// Forward.  Chunk c of `chunk` tokens is one CTA's; the part of it that lies
// in sequence q is summed into slot c + q (along the chunks and sequences that
// overlap, c + q takes each value once), so no sum needs an atomic and the
// order is fixed.  Three CTAs a SM is what the 32 running sums and 32 scores a lane
// leave room for.  16384 x 896 fp32 in 9 sequences: 23 us with the finish kernel
// (59 MB: 9 us at the copy rate), bf16 32; latency and issue (52%) bound it.
// ---------------------------------------------------------------------------
struct BalanceArgs {
    int T, n, k, S, chunk, nchunk;
    long long ld;
    const void* logits;
    const int32_t* idx;
    const int32_t* seq;
    const uint8_t* mask;
    float* part_p;     // [nchunk + S, n] sums of p
    int32_t* part_c;   // [nchunk + S, n] routes
    int32_t* part_t;   // [nchunk + S] valid tokens
    unsigned* ticket;  // [S]
    float* loss_part;  // [S, ceil(n / 32)]
    float* loss;
    int32_t* counts;
    float* probs;
    int32_t* tokens;
};

template <typename T, int V>
__global__ void __launch_bounds__(kBalThreads, 3) k_balance_partial(const BalanceArgs a) {
    pdl_trigger();
    extern __shared__ float sm[];
    float* red = sm;                                              // [kBalWarps][n]
    int* cnt = reinterpret_cast<int*>(sm + kBalWarps * a.n);      // [n]
    __shared__ int valid[kBalWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const T* logits = static_cast<const T*>(a.logits);
    const int c0 = blockIdx.x * a.chunk, c1 = min(a.T, c0 + a.chunk);
    if (blockIdx.x == 0)
        for (int q = threadIdx.x; q < a.S; q += kBalThreads) a.ticket[q] = 0;
    int q = a.seq ? find_seq(a.seq, a.S, c0) : 0;
    for (int t0 = c0; t0 < c1; ++q) {
        const int t1 = a.seq && q + 1 < a.S ? min(c1, max(t0, __ldg(a.seq + q + 1))) : c1;
        for (int j = threadIdx.x; j < a.n; j += kBalThreads) cnt[j] = 0;
        __syncthreads();
        float acc[kMaxPerLane] = {};
        int nv = 0;
        for (int t = t0 + warp; t < t1; t += kBalWarps) {
            if (a.mask && !__ldg(a.mask + t)) continue;
            ++nv;
            float x[kMaxPerLane];
            load_row<T, V>(logits + (long long)t * a.ld, a.n, lane, x);
            if (lane < a.k) {
                const int id = __ldg(a.idx + (long long)t * a.k + lane);
                if ((unsigned)id < (unsigned)a.n) atomicAdd(cnt + id, 1);
            }
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kMaxPerLane / V; ++i)
                if (32 * i * V < a.n) {   // uniform: groups past the row cost nothing
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        float e;
                        x[i * V + v] = (32 * i + lane) * V < a.n ? score(x[i * V + v], e) : 0.0f;
                        sum += x[i * V + v];
                    }
                }
            const float inv = 1.0f / warp_sum(sum);
#pragma unroll
            for (int i = 0; i < kMaxPerLane / V; ++i)
                if (32 * i * V < a.n) {
#pragma unroll
                    for (int v = 0; v < V; ++v) acc[i * V + v] = fmaf(x[i * V + v], inv, acc[i * V + v]);
                }
        }
#pragma unroll
        for (int i = 0; i < kMaxPerLane / V; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int j = (32 * i + lane) * V + v;
                if (j < a.n) red[warp * a.n + j] = acc[i * V + v];
            }
        if (lane == 0) valid[warp] = nv;
        __syncthreads();
        const long long slot = blockIdx.x + q;
        for (int j = threadIdx.x; j < a.n; j += kBalThreads) {
            float p = 0.0f;
#pragma unroll
            for (int w = 0; w < kBalWarps; ++w) p += red[w * a.n + j];
            a.part_p[slot * a.n + j] = p;
            a.part_c[slot * a.n + j] = cnt[j];
        }
        if (threadIdx.x == 0) {
            int tv = 0;
            for (int w = 0; w < kBalWarps; ++w) tv += valid[w];
            a.part_t[slot] = tv;
        }
        __syncthreads();
        t0 = t1;
    }
}

// CTA (q, b): experts 32 b .. 32 b + 31 of sequence q over its slots; the
// sequence's last CTA adds up its loss.
__global__ void __launch_bounds__(kBalThreads) k_balance_finish(const BalanceArgs a) {
    __shared__ float sp[kBalWarps][33];
    __shared__ int sc[kBalWarps][33];
    __shared__ int st[kBalWarps];
    __shared__ bool last;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int q = blockIdx.x, j = blockIdx.y * 32 + lane;
    pdl_wait();
    const int o0 = a.seq ? min(max(__ldg(a.seq + q), 0), a.T) : 0;
    const int o1 = a.seq ? min(max(__ldg(a.seq + q + 1), o0), a.T) : a.T;
    const int f = o0 / a.chunk, g = o1 > o0 ? (o1 - 1) / a.chunk + 1 : f;   // chunks [f, g)
    float p = 0.0f;
    int c = 0, t = 0;
    for (int u = f + warp; u < g; u += kBalWarps) {
        const long long slot = u + q;
        if (j < a.n) {
            p += a.part_p[slot * a.n + j];
            c += a.part_c[slot * a.n + j];
        }
        t += a.part_t[slot];
    }
    sp[warp][lane] = p;
    sc[warp][lane] = c;
    if (lane == 0) st[warp] = t;
    __syncthreads();
    if (warp == 0) {
        p = 0.0f, c = 0, t = 0;
        for (int w = 0; w < kBalWarps; ++w) p += sp[w][lane], c += sc[w][lane], t += st[w];
        const float inv_t = 1.0f / fmaxf((float)t, 1.0f);
        p *= inv_t;
        if (j < a.n) {
            a.probs[(long long)q * a.n + j] = p;
            a.counts[(long long)q * a.n + j] = c;
        }
        const float l = warp_sum(j < a.n ? (float)c * p : 0.0f) * ((float)a.n * inv_t / (float)a.k);
        if (lane == 0) {
            if (blockIdx.y == 0) a.tokens[q] = t;
            a.loss_part[(long long)q * gridDim.y + blockIdx.y] = l;
            __threadfence();
            last = atomicAdd(a.ticket + q, 1u) == gridDim.y - 1;
        }
        __syncwarp();
        if (last) {
            __threadfence();
            const float v = lane < (int)gridDim.y
                                ? *(volatile float*)(a.loss_part + (long long)q * gridDim.y + lane) : 0.0f;
            const float total = warp_sum(v);   // at most 32 CTAs a sequence
            if (lane == 0) a.loss[q] = total;
        }
    }
}

// ---------------------------------------------------------------------------
// Backward.  With f_j = dloss n counts_j / (k T_q^2), D = sum_j f_j p_j and the
// slope d_j = s_j c_j:
//   dx_j = d_j (f_j - D) / S_t                              balance loss
//        + d_j (dw_i - sum_l dw_l w_l) / sum_l s_(idx_l)    j = idx_i, mixture weights
// The slope is divided by the sum first: that quotient is at most 1, where the
// reciprocal of a sum alone reaches e^80.  Likewise D is summed over the counts (the
// factor of f after it) and the mean over weights, not scores: a score of e^-80 times
// a small gradient would be subnormal.
// A CTA has a chunk of tokens and the counts of the chunk's sequence in shared memory
// (a chunk that crosses a boundary goes through its sequences in turn).  A warp
// has its next row on the way to shared memory (cp.async) while it works on this
// one, where rows are 16-byte vectors.  The dense row is stored first, then the k
// chosen entries over it.  16384 x 896 fp32: 26 us (118 MB: 17 us at the copy rate),
// bf16 24, bound by issue (60%) as much as by memory; keeping more than the slopes in
// registers (fewer CTAs a SM, the chosen entries selected in the dense pass) took 83.
// ---------------------------------------------------------------------------
struct RouterGradArgs {
    int T, n, k, S, chunk;
    long long ld, ldg;
    const void* logits;
    const int32_t* idx;
    const int32_t* seq;
    const uint8_t* mask;
    const float* dw;
    const float* dloss;
    const int32_t* counts;
    const int32_t* tokens;
    void* out;
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src)
                 : "memory");
}

template <typename T, int V>
__global__ void __launch_bounds__(kBalThreads, 3) k_router_backward(const RouterGradArgs a) {
    extern __shared__ __align__(16) float fs[];   // [n rounded up to 8], then two rows a warp (V > 1)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    T* rows = reinterpret_cast<T*>(fs + ((a.n + 7) & ~7)) + (size_t)2 * warp * a.n;
    const int c0 = blockIdx.x * a.chunk, c1 = min(a.T, c0 + a.chunk);
    // this token's mask, and the expert and gradient of the lane's route
    auto scalars = [&](int t, bool& live, int& id, float& d) {
        live = t < c1 && (!a.mask || __ldg(a.mask + t));
        id = -1;
        d = 0.0f;
        if (a.dw && lane < a.k && t < c1) {
            id = __ldg(a.idx + (long long)t * a.k + lane);
            d = __ldg(a.dw + (long long)t * a.k + lane);
        }
    };
    auto fetch = [&](int t, int buf) {
        if constexpr (V > 1) {
            if (t < c1) {
                const T* row = static_cast<const T*>(a.logits) + (long long)t * a.ld;
                for (int j = lane * V; j < a.n; j += 32 * V) cp_async16(rows + buf * a.n + j, row + j);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    int q = a.dloss && a.seq ? find_seq(a.seq, a.S, c0) : 0;
    // The warp's tokens c0 + warp, c0 + warp + 8, ... in turn, whatever their sequence.
    int t = c0 + warp, buf = 0;
    bool live;
    int id;
    float d;
    fetch(t, buf);
    scalars(t, live, id, d);
    float scale = 0.0f;   // f_j = scale counts_j
    for (int t0 = c0; t0 < c1; ++q) {
        const int t1 = a.dloss && a.seq && q + 1 < a.S ? min(c1, max(t0, __ldg(a.seq + q + 1))) : c1;
        if (t1 > t0) {
            __syncthreads();   // the last sequence's readers are done
            scale = 0.0f;
            if (a.dloss) {
                const float tq = fmaxf((float)__ldg(a.tokens + q), 1.0f);
                scale = __ldg(a.dloss + q) * ((float)a.n / ((float)a.k * tq)) / tq;
            }
            for (int j = threadIdx.x; j < a.n; j += kBalThreads)
                fs[j] = a.dloss ? (float)__ldg(a.counts + (long long)q * a.n + j) : 0.0f;
            __syncthreads();
        }
        for (; t < t1; t += kBalWarps, buf ^= 1) {
            const T* row = static_cast<const T*>(a.logits) + (long long)t * a.ld;
            T* out = static_cast<T*>(a.out) + (long long)t * a.ldg;
            fetch(t + kBalWarps, buf ^ 1);
            bool next_live;
            int next_id;
            float next_d;
            scalars(t + kBalWarps, next_live, next_id, next_d);
            if constexpr (V > 1) {
                asm volatile("cp.async.wait_group 1;" ::: "memory");
                __syncwarp();
                row = rows + buf * a.n;
            }
            if (!live) {
                for (int j = lane; j < a.n; j += 32) out[j] = from_f32<T>(0.0f);
            } else {
                // the chosen experts, one a lane
                float own = 0.0f, slope = 0.0f;
                const bool chosen = (unsigned)id < (unsigned)a.n;
                if (chosen) own = score_slope(to_f32<T>(row[id]), slope);
                else d = 0.0f;
                float x[kMaxPerLane];   // the row, then its slopes
                if (V == 1) load_row<T, V>(row, a.n, lane, x);
                float sum = 0.0f, dot = 0.0f;
#pragma unroll
                for (int i = 0; i < kMaxPerLane / V; ++i) {
                    const int j = (32 * i + lane) * V;
                    if (j >= a.n) continue;
                    float f[V];
                    if constexpr (V == 1) {
                        f[0] = fs[j];
                    } else {
#pragma unroll
                        for (int u = 0; u < V / 4; ++u)
                            *reinterpret_cast<float4*>(f + 4 * u) = *reinterpret_cast<const float4*>(fs + j + 4 * u);
                        const uint4 u = *reinterpret_cast<const uint4*>(row + j);
#pragma unroll
                        for (int v = 0; v < V; ++v) x[i * V + v] = to_f32<T>(reinterpret_cast<const T*>(&u)[v]);
                    }
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        float sl;
                        const float s = score_slope(x[i * V + v], sl);
                        x[i * V + v] = sl;
                        sum += s;
                        dot = fmaf(f[v], s, dot);
                    }
                }
                // without a balance loss the scores of the others are not part of the gradient (nor a NaN there)
                const float inv = a.dloss ? 1.0f / warp_sum(sum) : 0.0f;
                const float D = a.dloss ? scale * (warp_sum(dot) * inv) : 0.0f;
                float w_inv = 0.0f, mean = 0.0f;
                if (a.dw) {
                    const float all = warp_sum(own);
                    w_inv = all > 0.0f ? 1.0f / all : all != all ? all : 0.0f;
                    mean = warp_sum(d * (own * w_inv));
                }
#pragma unroll
                for (int i = 0; i < kMaxPerLane / V; ++i) {
                    const int j = (32 * i + lane) * V;
                    if (j >= a.n) continue;
                    if constexpr (V == 1) {
                        out[j] = from_f32<T>((x[i] * inv) * fmaf(fs[j], scale, -D));
                    } else {
                        float f[V];
#pragma unroll
                        for (int u = 0; u < V / 4; ++u)
                            *reinterpret_cast<float4*>(f + 4 * u) = *reinterpret_cast<const float4*>(fs + j + 4 * u);
                        uint4 o;
                        T* e = reinterpret_cast<T*>(&o);
#pragma unroll
                        for (int v = 0; v < V; ++v) e[v] = from_f32<T>((x[i * V + v] * inv) * fmaf(f[v], scale, -D));
                        *reinterpret_cast<uint4*>(out + j) = o;
                    }
                }
                if (a.dw) {
                    __syncwarp();   // the row is stored before the chosen entries
                    if (chosen)
                        out[id] = from_f32<T>(fmaf(slope * inv, fmaf(fs[id], scale, -D), (slope * w_inv) * (d - mean)));
                }
            }
            __syncwarp();   // the row's readers are done before its buffer is filled again
            live = next_live;
            id = next_id;
            d = next_d;
        }
        t0 = t1;
    }
}

// Tokens per CTA: one wave of `ctas` a SM at full size (what the registers
// allow), one token a warp at least.
int chunk_of(int T, int ctas) {
    const int per = (T + 152 * ctas - 1) / (152 * ctas);
    return ((per + kBalWarps - 1) / kBalWarps) * kBalWarps;
}
int balance_chunk(int T) { return chunk_of(T, 3); }

struct BalanceLayout {
    size_t part_p, part_c, part_t, ticket, loss_part, total;
};
BalanceLayout balance_layout(int T, int n, int S) {
    const size_t slots = (size_t)((T + balance_chunk(T) - 1) / balance_chunk(T)) + S;
    BalanceLayout l;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = qbh::align_up(off + bytes, 256);
        return o;
    };
    l.part_p = take(slots * n * 4);
    l.part_c = take(slots * n * 4);
    l.part_t = take(slots * 4);
    l.ticket = take((size_t)S * 4);
    l.loss_part = take((size_t)S * ((n + 31) / 32) * 4);
    l.total = off;
    return l;
}

bool router_sizes_ok(int T, int n, int k, int S, int dtype, long long ld) {
    return T >= 1 && T <= QBMOE_MAX_ROWS && n >= 2 && n <= QBMOE_MAX_EXPERTS && k >= 1 && k <= n && k <= QBMOE_MAX_TOPK && S >= 1 &&
           S <= QBMOE_MAX_ROWS && (dtype == QBMOE_F32 || dtype == QBMOE_BF16) && ld >= n;
}
bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Rows are read as 16-byte vectors when every row starts on one.
template <typename T>
bool vector_rows(int n, const void* p, long long ld) {
    return n % Vec<T>::n == 0 && ld % Vec<T>::n == 0 && qbh::aligned16(p);
}

}  // namespace

int qbh::balance_init() {
    const int most = QBMOE_MAX_EXPERTS * 4 * (1 + 2 * kBalWarps);
    int rc = cuda_err(cudaFuncSetAttribute(k_router_backward<float, 4>, cudaFuncAttributeMaxDynamicSharedMemorySize, most));
    if (!rc)
        rc = cuda_err(cudaFuncSetAttribute(k_router_backward<__nv_bfloat16, 8>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, most));
    return rc;
}

extern "C" size_t qbmoe_balance_workspace_bytes(int T, int n, int S) {
    if (T < 1 || T > QBMOE_MAX_ROWS || n < 2 || n > QBMOE_MAX_EXPERTS || S < 1 || S > QBMOE_MAX_ROWS) return 0;
    return balance_layout(T, n, S).total;
}

extern "C" int moe_balance_loss(int T, int n, int k, int S, int logit_dtype, const void* logits, long long ld,
                                const int32_t* idx, const int32_t* seq_offsets, const uint8_t* token_mask,
                                float* loss, int32_t* counts, float* probs, int32_t* tokens, void* workspace,
                                size_t workspace_bytes, qbmoe_stream_t stream) {
    if (!router_sizes_ok(T, n, k, S, logit_dtype, ld)) return QBMOE_EINVAL;
    if (!logits || !idx || !loss || !counts || !probs || !tokens || !workspace) return QBMOE_EINVAL;
    if (!seq_offsets && S != 1) return QBMOE_EINVAL;
    const size_t es = logit_dtype == QBMOE_BF16 ? 2 : 4;
    if (!aligned_to(logits, es)) return QBMOE_EINVAL;
    for (const void* p : {(const void*)idx, (const void*)seq_offsets, (const void*)loss, (const void*)counts,
                          (const void*)probs, (const void*)tokens})
        if (p && !aligned_to(p, 4)) return QBMOE_EINVAL;
    if (!aligned_to(workspace, 256)) return QBMOE_EINVAL;
    const BalanceLayout l = balance_layout(T, n, S);
    if (workspace_bytes < l.total) return QBMOE_EWORKSPACE;
    int rc = qbh::device_init();
    if (rc) return rc;
    char* ws = static_cast<char*>(workspace);
    BalanceArgs a{};
    a.T = T; a.n = n; a.k = k; a.S = S; a.ld = ld;
    a.chunk = balance_chunk(T);
    a.nchunk = (T + a.chunk - 1) / a.chunk;
    a.logits = logits; a.idx = idx; a.seq = seq_offsets; a.mask = token_mask;
    a.part_p = reinterpret_cast<float*>(ws + l.part_p);
    a.part_c = reinterpret_cast<int32_t*>(ws + l.part_c);
    a.part_t = reinterpret_cast<int32_t*>(ws + l.part_t);
    a.ticket = reinterpret_cast<unsigned*>(ws + l.ticket);
    a.loss_part = reinterpret_cast<float*>(ws + l.loss_part);
    a.loss = loss; a.counts = counts; a.probs = probs; a.tokens = tokens;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const size_t smem = (size_t)(kBalWarps + 1) * n * 4;   // at most 36 KB
    if (logit_dtype == QBMOE_F32) {
        if (vector_rows<float>(n, logits, ld)) k_balance_partial<float, 4><<<a.nchunk, kBalThreads, smem, s>>>(a);
        else k_balance_partial<float, 1><<<a.nchunk, kBalThreads, smem, s>>>(a);
    } else {
        if (vector_rows<__nv_bfloat16>(n, logits, ld))
            k_balance_partial<__nv_bfloat16, 8><<<a.nchunk, kBalThreads, smem, s>>>(a);
        else k_balance_partial<__nv_bfloat16, 1><<<a.nchunk, kBalThreads, smem, s>>>(a);
    }
    if ((rc = qbh::cuda_err(cudaGetLastError()))) return rc;
    return qbh::launch_pdl(k_balance_finish, dim3(S, (n + 31) / 32), dim3(kBalThreads), 0, s, a);
}

extern "C" int moe_router_backward(int T, int n, int k, int S, int logit_dtype, const void* logits, long long ld,
                                   const int32_t* idx, const int32_t* seq_offsets, const uint8_t* token_mask,
                                   const float* dw, const float* dloss, const int32_t* counts,
                                   const int32_t* tokens, void* dlogits, long long ldg, qbmoe_stream_t stream) {
    if (!router_sizes_ok(T, n, k, S, logit_dtype, ld) || ldg < n) return QBMOE_EINVAL;
    if (!logits || !idx || !dlogits || (!dw && !dloss)) return QBMOE_EINVAL;
    if (dloss ? (!counts || !tokens) : (counts || tokens)) return QBMOE_EINVAL;
    if (!seq_offsets && S != 1) return QBMOE_EINVAL;
    if (dlogits == logits && ldg != ld) return QBMOE_EINVAL;
    const size_t es = logit_dtype == QBMOE_BF16 ? 2 : 4;
    if (!aligned_to(logits, es) || !aligned_to(dlogits, es)) return QBMOE_EINVAL;
    for (const void* p : {(const void*)idx, (const void*)seq_offsets, (const void*)dw, (const void*)dloss,
                          (const void*)counts, (const void*)tokens})
        if (p && !aligned_to(p, 4)) return QBMOE_EINVAL;
    int rc = qbh::device_init();
    if (rc) return rc;
    RouterGradArgs a{};
    a.T = T; a.n = n; a.k = k; a.S = S; a.ld = ld; a.ldg = ldg;
    a.logits = logits; a.idx = idx; a.seq = seq_offsets; a.mask = token_mask;
    a.dw = dw; a.dloss = dloss; a.counts = counts; a.tokens = tokens; a.out = dlogits;
    a.chunk = chunk_of(T, 3);
    const int grid = (T + a.chunk - 1) / a.chunk;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const size_t fbytes = (size_t)((n + 7) & ~7) * 4, rbytes = (size_t)2 * kBalWarps * n * es;   // at most 68 KB
    if (logit_dtype == QBMOE_F32) {
        if (vector_rows<float>(n, logits, ld) && vector_rows<float>(n, dlogits, ldg))
            k_router_backward<float, 4><<<grid, kBalThreads, fbytes + rbytes, s>>>(a);
        else k_router_backward<float, 1><<<grid, kBalThreads, fbytes, s>>>(a);
    } else {
        if (vector_rows<__nv_bfloat16>(n, logits, ld) && vector_rows<__nv_bfloat16>(n, dlogits, ldg))
            k_router_backward<__nv_bfloat16, 8><<<grid, kBalThreads, fbytes + rbytes, s>>>(a);
        else k_router_backward<__nv_bfloat16, 1><<<grid, kBalThreads, fbytes, s>>>(a);
    }
    return qbh::cuda_err(cudaGetLastError());
}
