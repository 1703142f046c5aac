// What the MXFP4 products share: grouped tiles, tensor maps, the status word.
#pragma once

#include "common.cuh"

#include <cuda.h>

namespace qbh {

// Kernel attributes, once per device (device_init).
int mx_product_init();   // mxfp4_product.cu
int mx_grad_init();      // mxfp4_grad.cu
int matvec_init();       // matvec.cu
int experts_init();      // experts.cu
int rmsnorm_init();      // rmsnorm.cu
int pieces_init();       // pieces.cu

// Expired waits of the calls that take no context, counted on each device; and, after
// synchronising s, whether there were any since the calling thread last asked
// (QBMOE_OK or QBMOE_ETIMEOUT).
int* mx_expiries();
int mx_new_expiries(cudaStream_t s);
// Test hooks of those calls (qbmoe_set_wait_limit / qbmoe_debug_stall without a
// context), for the calls that the same host thread makes.
long long mx_wait_limit();
void mx_set_wait_limit(long long polls);
int mx_stall();
void mx_set_stall(int on);

int sm_count();
// 2-D row-major tensor map: cols elements a row (row stride ld bytes), box
// {box_cols, box_rows}, zeros outside; swizzled over the box's 128 bytes, or 64 of
// codes, unless `plain`.
bool encode_rows(CUtensorMap* m, CUtensorMapDataType type, const void* base, long long rows, long long cols,
                 long long ld_bytes, int box_cols, int box_rows, bool plain = false);

// Rows of fp32 or bf16 (x_type) to codes and scales, and the values if wanted (mxfp4.cu).
int mx_quantize(long long rows, int K, int x_type, const void* x, long long ldx, uint8_t* codes, uint8_t* scales,
                void* values, cudaStream_t s);

// Sizes and alignment are checked by the caller.  raw: rows of another type
// that are quantised into x_codes and x_scales first (NULL: they hold the rows).
struct MxProduct {
    int R, E, N, K;
    uint8_t *x_codes, *x_scales;
    const uint8_t *w_codes, *w_scales;
    const int32_t* offsets;
    void* y;
    long long ldy;
    const void* raw;
    int raw_type;
    long long raw_ld;
};
int mx_product(const MxProduct& p, cudaStream_t s);

// dx (codes and scales of the weights) or dw (of the rows) from dy [R, N] bf16.
struct MxGrad {
    bool weights;
    int R, E, N, K;
    const void* dy;
    long long lddy;
    const uint8_t *codes, *scales;
    const int32_t* offsets;
    void* out;
    long long ldo;
    int out_type;
    void* parts;   // dw in parts: fp32 [splits, E, N, K], NULL for one part
};
int mx_grad(const MxGrad& g, cudaStream_t s);
int mx_wgrad_splits(int R, int E, int N, int K);

}  // namespace qbh

namespace qb {

// Expert-ordered rows as tiles of at most BN rows: seg [E + 1] and toff [E + 1]
// (first tile of each expert) in shared memory.  Offsets out of order or out
// of range are clamped, so that every tile lies inside [0, R).
struct Groups {
    int* seg;
    int* toff;
};

// Whole CTA: read the offsets and count each expert's tiles.  NULL offsets: one
// group of R rows.  Ends with a __syncthreads.
template <int BN, int kThreads>
QB_DEV void load_groups(const Groups& g, const int32_t* offsets, int E, int R, int* scratch /* [kThreads / 32] */) {
    constexpr int kWarps = kThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e <= E; e += kThreads)
        g.seg[e] = offsets ? min(max(__ldcg(offsets + e), 0), R) : (e ? R : 0);
    __syncthreads();
    // each warp scans a run of experts, then adds what the warps before it counted
    const int per = ((E + kWarps - 1) / kWarps + 31) & ~31;
    int run = 0;
    for (int e0 = warp * per; e0 < min(E, (warp + 1) * per); e0 += 32) {
        const int e = e0 + lane;
        int n = e < E ? (max(g.seg[e + 1] - g.seg[e], 0) + BN - 1) / BN : 0;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (e < E) g.toff[e] = run + incl - n;
        run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) scratch[warp] = run;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += scratch[w];
    for (int e = warp * per + lane; e < min(E, (warp + 1) * per); e += 32) g.toff[e] += before;
    if (threadIdx.x == 0) {
        int total = 0;
        for (int w = 0; w < kWarps; ++w) total += scratch[w];
        g.toff[E] = total;
    }
    __syncthreads();
}

// Walks the tiles blockIdx.x, blockIdx.x + gridDim.x, ... of a grid whose m
// index is fastest, then the row tiles of all experts.  Every lane of the warp
// calls.  Lane l holds what the tiles of expert base + l need, so a step is a
// ballot and three shuffles; shared memory (whose latency is several hundred
// cycles while the tensor cores stream their operands from it) is read once
// per 32 experts.  An expert's rows are split into equal tiles (multiples of
// 16), so that tiles sharing a weight tile run at one pace.
template <int BN>
struct Walker {
    int ntg, m, g;
    int row0, nrows;              // of the current tile
    int base, w_first, w_next, w_row, w_end, w_per;   // this lane's expert: tiles [first, next), rows, rows a tile
    int total;
    QB_DEV void window(const Groups& gr, int E, int from) {
        base = from;
        const int e = min(from + (int)(threadIdx.x & 31), E - 1);
        const bool past = from + (int)(threadIdx.x & 31) >= E;
        w_first = gr.toff[e];
        w_next = past ? 0x7fffffff : gr.toff[e + 1];
        w_row = gr.seg[e];
        w_end = gr.seg[e + 1];
        const int len = w_end - w_row, nt = max(w_next - w_first, 1);
        w_per = ((nt == 1 || past ? len : (len + nt - 1) / nt) + 15) & ~15;
    }
    QB_DEV void seek(const Groups& gr, int E) {   // ntg < total
        unsigned le;
        while ((le = __ballot_sync(0xffffffffu, w_next <= ntg)) == 0xffffffffu) window(gr, E, base + 32);
        const int i = __popc(le);   // toff never falls: the lanes that pass come first
        g = base + i;
        const int per = __shfl_sync(0xffffffffu, w_per, i), t0 = __shfl_sync(0xffffffffu, w_first, i);
        row0 = __shfl_sync(0xffffffffu, w_row, i) + (ntg - t0) * per;
        nrows = min(per, __shfl_sync(0xffffffffu, w_end, i) - row0);
    }
    QB_DEV void start(const Groups& gr, int E, int m_total) {
        total = gr.toff[E];
        ntg = blockIdx.x / m_total;
        m = blockIdx.x - ntg * m_total;
        window(gr, E, 0);
        if (ntg < total) seek(gr, E);
    }
    QB_DEV void next(const Groups& gr, int E, int m_total) {
        const int was = ntg;
        m += gridDim.x;
        while (m >= m_total) m -= m_total, ++ntg;
        if (ntg != was && ntg < total) seek(gr, E);
    }
};

}  // namespace qb
