// MXFP4 weights streamed past a few rows: what moe_mxfp4_matvec and moe_mxfp4_experts share for small calls
// and for depths that pieces.cuh does not take.
//
// One kernel brings weights through shared memory and multiplies them with a few rows that
// stay in registers (more than fit: with over 8 blocks a warp its variants store 12 to 280 bytes a thread on the
// stack).  A persistent CTA a SM takes a contiguous run of units; a unit is kMT
// tiles of 16 weight rows over the whole depth (or one slab of it).  Eight consumer warps of 168 registers
// form groups that take units in turn, so that one group's fixed work per unit falls into another's products
// (sixteen warps of 96 registers, one tile a unit: 413 against 408 us by 896 experts of 1024 x 3584, and 4096 rows'
// whole experts 1524 against 1370; twelve warps 430 and 1862).  The warps of a group divide the depth: a
// warp owns a run of kNB blocks of 32 of K, for which it holds the rows' elements as mma B
// operands, so that the rows cost no bandwidth while weights go by.  Per block of 32 and tile:
//   - ldmatrix hands each quad of lanes the 16 bytes of a weight row's block;
//   - codes become fp16 (exact) two at a time, with one conversion;
//   - two m16n8k16 products, weights as A (16 rows), 8 columns of x as B (for the SiTU-GLU's fp32 results two more, of
//     what fp16 leaves of them: with half as many blocks a warp, 256 tokens' 16 routes over 896 experts of 3552 / 992
//     take 1484 us, with one term and all blocks 1587, with the second term in columns of its own 2071);
//   - the block's dot products, times the two scales, are added in fp32.
// Two producer warps, a stage each in turn, bring codes (long rows one by one, short ones
// in TMA boxes: a copy costs 20 to 80 cycles to issue) and scales several units ahead; two more
// add the consumers' shares of the depth, in order, and store.
// Weight rows are the M operand of the small mma because a column costs nothing that way: up
// to 8 rows of x take as long as one.
//
// Measured (GPU time, cold caches): one row by 6144 x 7168 24 us (the weights alone take 3.5; 19 with part of them in
// L2), by 12288 x 7168 30; 13 rows by 896 x 7168 16, 10 from L2 for a floor of 0.5: route lists and barriers, rows to
// registers and code fetched cold come before the first product.  A large call spends 74 cycles a scheduler on a block
// and tile (the products' own
// instructions take 35, HBM 46): waits, sums and scales of each unit; pieces.cuh has those.
#pragma once

#include "mxfp4.cuh"
#include "mxfp4_decode.cuh"
#include "tc_ptx.cuh"

#include <cuda_fp16.h>

#include <initializer_list>

namespace {

using namespace qb;

constexpr int kWarps = 8;                      // consumers; then two producers and two that sum
constexpr int kThreads = 32 * (kWarps + 4);    // 168 registers a thread
constexpr int kCols = 8;                       // rows of x a unit takes
constexpr int kMaxStages = 32;
constexpr int kLine = 20;                      // floats a column of 16 results takes: stores without bank conflicts
constexpr long long kDefaultWait = 1LL << 17;  // polls (<= 20 us each) before a wait expires
constexpr int kMaxDynamic = 226 * 1024;       // of 227 KB, a little being static
constexpr int kSlack = 128;                    // scales are read by the word, up to 8 bytes ahead

// What a launch computes.
enum { kStore, kGlu, kDown };
// fp16 terms of an element of x: the SiTU-GLU's fp32 results take two, the second of what the first leaves (together
// within 2^-22 of the value), in half as many blocks a warp.
constexpr int terms_of(int mode) { return mode == kDown ? 2 : 1; }
constexpr int kBox = 8;                        // blocks of 32 in a row of a TMA box: 128 bytes of codes

struct StreamArgs {
    int R, E, N, K;              // rows of x, experts, weight rows (features of kGlu), depth
    int x_type;
    const void* x;               // kDown: fp32 [R, K]
    long long ldx;
    const uint8_t* x_scales;
    CUtensorMap codes, codes2;           // [E N, K / 2] bytes; kGlu: gate and up
    const uint8_t *w, *w2;               // the same, for copies of single rows
    const uint8_t *scales, *scales2;     // [E, N, K / 32]
    const int32_t* offsets;      // kStore: [E + 1] or NULL
    const int32_t* idx;          // kGlu, kDown: routes [R]
    int k;                       // kGlu: routes a token
    int y_type;
    void* y;                     // [slabs, R, N]; kGlu: fp32 [R, N], in slabs fp32 [slabs, 2, R, N]; kDown: fp32
    long long ldy;
    float beta1, beta2;
    // geometry
    int splits, groups;          // consumers along the depth: a group; kWarps / splits of them
    int slabs, slab_blocks;      // the depth in slabs of this many blocks of 32
    int stages, stage_bytes;
    int pitch;                   // bytes between the rows of a unit that come one by one; 0: they come in boxes
    int rows;                    // scales of a unit come row by row (slabs), else all together
    int scale_pitch;             // bytes between the scales of its rows
    int* expiries;
    long long wait_limit;
    int stall;
};

// kNB blocks of 32 a warp, kMT tiles a unit; weights come in boxes, a whole number a warp, or row by row.
template <int kNB, int kMT, bool kBoxed>
struct Shape {
    static constexpr int kBlocks = kNB, kTiles = kMT;
    static constexpr bool kBoxes = kBoxed;
    static constexpr int kStaged = kBoxes ? kMT : 1;           // tiles a stage
    static constexpr int kPart = kCols * kLine + 8;            // floats of a warp's partial results
    static constexpr int kRed = 2 * kWarps * kMT * kPart * 4;  // two slots a group
    static constexpr int kSx = kWarps * kNB * kCols * 4;       // scales of x
    static constexpr int kBars = (2 * kMaxStages + 4 * kWarps) * 8;
    // before the ring, which starts at a multiple of 1024
    static size_t fixed(int E, int routes) {   // bytes
        return kBars + kRed + kSx + qbh::align_up((size_t)(E + 1) * 8, 16) + (size_t)routes * 2 + 1024;
    }
};

QB_DEV void codes_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
// d = A B
QB_DEV void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// d += A B
QB_DEV void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
QB_DEV void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
QB_DEV uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
// Two E8M0 bytes of a word, the low two or the high two, as fp32 (0xFF: NaN).
QB_DEV void scale_pair(uint32_t word, bool high, float& a, float& b) {
    uint32_t h;
    if (high) asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.bf16x2.ue8m0x2 %0, u;\n\t}" : "=r"(h) : "r"(word));
    else asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.bf16x2.ue8m0x2 %0, l;\n\t}" : "=r"(h) : "r"(word));
    a = __uint_as_float(h << 16);
    b = __uint_as_float(h & 0xffff0000u);
}
// (a x, b y), in one instruction.
QB_DEV float2 mul2(float a, float b, float2 v) {
    float2 r;
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\t"
        "mul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a), "f"(b), "f"(v.x), "f"(v.y));
    return r;
}
QB_DEV void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
                 : "memory");
}

// ---------------------------------------------------------------------------
// Rows of x as B operands.  Lane 4 c + t holds elements 8 t .. 8 t + 7 of column c's block:
// the same share of K that ldmatrix gives lane 4 r + t of weight row r, so that the
// products pair the right elements.
// ---------------------------------------------------------------------------
QB_DEV uint32_t f16_pair(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
// A block whose largest magnitude m has these fp32 bits, as fp16: its largest element is put
// into [2^15, 65504], so that a bf16 element is exact down to 2^-32 of it, and smaller ones are within
// 2^-40 of it.  A block with an infinity or a NaN keeps those alone, which decide the result.
// kTerms 2: pairs 4 to 7 hold what the first four leave of the elements, in the same unit: both within 2^-22 of an
// element, or 2^-40 of the largest.
template <int kTerms>
QB_DEV float block_to_f16(const float (&v)[8], uint32_t m, uint32_t (&b)[4 * kTerms]) {
    const int ef = max((int)((m + 0x1000u) >> 23), 16);   // of m rounded to fp16's 11 bits
    const bool bad = m >= 0x7f800000u;
    const float inv = __int_as_float((269 - ef) << 23);   // 2^(15 - exponent); not used when bad
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float p = v[2 * j] * inv, q = v[2 * j + 1] * inv;
        if (bad) {
            p = (__float_as_uint(v[2 * j]) & 0x7f800000u) == 0x7f800000u ? v[2 * j] : 0.0f;
            q = (__float_as_uint(v[2 * j + 1]) & 0x7f800000u) == 0x7f800000u ? v[2 * j + 1] : 0.0f;
        }
        b[j] = f16_pair(p, q);
        if (kTerms == 2) {
            const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&b[j]));
            b[4 + j] = bad ? 0u : f16_pair(p - h.x, q - h.y);   // (exact differences)
        }
    }
    return bad ? 1.0f : __int_as_float((ef - 15) << 23);
}
// This lane's 8 elements of a block as they are stored: 16 bytes of bf16, 8 of E4M3 and a
// scale byte, or 32 of fp32.
template <int kX>
struct Raw {
    uint4 u, v;
    QB_DEV void load(const StreamArgs& a, long long row, int blk, bool have) {
        const int at = blk * 32 + 8 * (threadIdx.x & 3);
        u = v = make_uint4(0, 0, 0, 0);
        if (!have) return;
        if (kX == QBMOE_MXFP8) {
            const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.x) + row * a.ldx + at);
            u.x = q.x;
            u.y = q.y;
            u.z = a.x_scales[row * (a.K >> 5) + blk];
        } else if (kX == QBMOE_F32) {   // from the kernel before
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(a.x) + row * a.ldx + at);
            u = __ldcg(p);
            v = __ldcg(p + 1);
        } else {
            u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.x) + row * a.ldx + at);
        }
    }
    // The four pairs of fp16 a term and (in every lane of the quad) the block's scale.
    template <int kTerms>
    QB_DEV float convert(uint32_t (&b)[4 * kTerms]) const {
        if (kX == QBMOE_MXFP8) {
            asm("{\n\t.reg .b16 p, q, r, s;\n\tmov.b32 {p, q}, %4;\n\tmov.b32 {r, s}, %5;\n\t"
                "cvt.rn.f16x2.e4m3x2 %0, p;\n\tcvt.rn.f16x2.e4m3x2 %1, q;\n\t"
                "cvt.rn.f16x2.e4m3x2 %2, r;\n\tcvt.rn.f16x2.e4m3x2 %3, s;\n\t}"
                : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                : "r"(u.x), "r"(u.y));
            return e8m0_value(u.z);
        }
        float f[8];
        const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f[j] = __uint_as_float(kX == QBMOE_F32 ? w[j] : j & 1 ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7fffffffu);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        return block_to_f16<kTerms>(f, m, b);
    }
};

// ---------------------------------------------------------------------------
// Which rows belong together.
// ---------------------------------------------------------------------------

// Whole CTA: a[0 .. n - 1] to its exclusive sums, the total in a[n].
QB_DEV void exclusive_scan(int* a, int n, int* scratch /* [kThreads / 32] */) {
    constexpr int W = kThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = ((n + W - 1) / W + 31) & ~31;
    __syncthreads();
    int run = 0;
    for (int i0 = warp * per; i0 < min(n, (warp + 1) * per); i0 += 32) {
        const int v = i0 + lane < n ? a[i0 + lane] : 0;
        int incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        if (i0 + lane < n) a[i0 + lane] = run + incl - v;
        run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) scratch[warp] = run;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < W; ++w) {
        if (w < warp) before += scratch[w];
        total += scratch[w];
    }
    for (int i = warp * per + lane; i < min(n, (warp + 1) * per); i += 32) a[i] += before;
    if (threadIdx.x == 0) a[n] = total;
    __syncthreads();
}

// seg [E + 1]: first row of each expert (kGlu, kDown: place in list, the routes in expert
// order); first [E + 1]: its first chunk of kCols rows.  Offsets out of order or out of
// range are clamped, so that every chunk lies inside [0, R).  Every CTA makes the same list, in the
// order of the routes: hist [warps][E] (in the ring, which nothing uses yet) counts each
// warp's share of them.
template <int kMode>
QB_DEV void group_rows(const StreamArgs& a, int* seg, int* first, uint16_t* list, int* hist, int* scratch) {
    if (kMode == kGlu || kMode == kDown) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const int warps = min(8, (a.R + 31) >> 5), per = ((a.R + warps - 1) / warps + 31) & ~31;
        for (int i = threadIdx.x; i < warps * a.E; i += kThreads) hist[i] = 0;
        __syncthreads();
        for (int r = warp * per + lane; r < min(a.R, (warp + 1) * per) && warp < warps; r += 32) {
            const int e = __ldg(a.idx + r);
            if (e >= 0 && e < a.E) atomicAdd(hist + warp * a.E + e, 1);
        }
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += kThreads) {
            int n = 0;
            for (int w = 0; w < warps; ++w) {
                const int c = hist[w * a.E + e];
                hist[w * a.E + e] = n;
                n += c;
            }
            seg[e] = n | ((n + kCols - 1) / kCols) << 16;   // both sums at once: at most 4096 routes, and no more chunks
        }
        exclusive_scan(seg, a.E, scratch);
        for (int e = threadIdx.x; e <= a.E; e += kThreads) {
            const int both = seg[e];
            first[e] = both >> 16;
            seg[e] = both & 0xffff;
        }
        __syncthreads();
        for (int r0 = warp * per; r0 < min(a.R, (warp + 1) * per) && warp < warps; r0 += 32) {
            const int r = r0 + lane, e = r < a.R ? __ldg(a.idx + r) : -1;
            const bool route = e >= 0 && e < a.E;
            const uint32_t same = __match_any_sync(0xffffffffu, route ? e : -1), before = same & ((1u << lane) - 1);
            int at = 0;
            if (route) {
                at = hist[warp * a.E + e];
                list[seg[e] + at + __popc(before)] = (uint16_t)r;
            }
            __syncwarp();
            if (route && !before) hist[warp * a.E + e] = at + __popc(same);
            __syncwarp();
        }
        tc::fence_proxy_async_smem();   // bulk copies write the ring next
        __syncthreads();
    } else if (!a.offsets) {
        if (threadIdx.x == 0) seg[0] = 0, seg[1] = a.R, first[0] = 0, first[1] = (a.R + kCols - 1) / kCols;
        __syncthreads();
    } else {
        for (int e = threadIdx.x; e <= a.E; e += kThreads) seg[e] = min(max(__ldg(a.offsets + e), 0), a.R);
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += kThreads) first[e] = (max(seg[e + 1] - seg[e], 0) + kCols - 1) / kCols;
        exclusive_scan(first, a.E, scratch);
    }
}

// Walks this CTA's run of units: tiles fastest, then chunks of rows, then slabs of the depth.
struct Units {
    long long u, end;
    int tile, tiles, chunk, chunks, slab;
    int g;                 // expert of the chunk
    bool fresh;            // the rows changed
    QB_DEV void start(const int* first, int E, int tiles_, int slabs) {
        tiles = tiles_;
        chunks = first[E];
        const long long total = (long long)chunks * tiles * slabs;
        u = total * blockIdx.x / gridDim.x;
        end = total * (blockIdx.x + 1) / gridDim.x;
        if (u >= end) return;
        tile = (int)(u % tiles);
        const long long c = u / tiles;
        chunk = (int)(c % chunks);
        slab = (int)(c / chunks);
        g = 0;             // the last expert whose first chunk is not behind this one
        for (int hi = E; hi - g > 1;) {
            const int mid = (g + hi) >> 1;
            if (first[mid] <= chunk) g = mid; else hi = mid;
        }
        fresh = true;
    }
    // Goes on by n units.
    QB_DEV void next(const int* first, int n = 1) {
        u += n;
        fresh = false;
        if ((tile += n) < tiles || u >= end) return;
        fresh = true;
        while (tile >= tiles) {
            tile -= tiles;
            if (++chunk == chunks) chunk = 0, ++slab, g = 0;
            while (first[g + 1] <= chunk) ++g;
        }
    }
};

// A warp's share of kMT tiles: each 16 weight rows times kNB blocks of K.  wat: this lane's row of the
// four 8 x 16-byte matrices that an ldmatrix loads (two blocks of 16 rows), of every of the first four
// loads in a box, whose 16-byte pieces are swizzled, else of the first alone; `at`: where each tile's
// stage lies; lo, hi: the scales of its weight rows lane / 4 and 8 more.  kSome: only nb blocks are the
// warp's; for the rest B and the scales of x are zeros, and the weights' scales, whatever lies there, are
// cleared lest one be NaN.
template <int kNB, int kMT, bool kBoxes, bool kSome, int kTerms>
QB_DEV void share(const uint32_t (&B)[kNB][4 * kTerms], const float* sx, const uint32_t (&wat)[4], const uint32_t (&at)[kMT],
                  const uint32_t (&lo)[kMT], const uint32_t (&hi)[kMT], int nb, float (&acc)[kMT][4]) {
    constexpr int box_bytes = 16 * kMT * 128;   // (boxes hold all tiles of a unit)
    auto load = [&](uint32_t (&w)[4], int i, int m) { ldmatrix4(w, (kBoxes ? wat[i / 2 % 4] + i / kBox * box_bytes : wat[0] + i * 16) + at[m]); };
    uint32_t sat[kMT][2], shift[kMT][2], sw[kMT][2], sc[kMT][2], next[kMT][4];
#pragma unroll
    for (int m = 0; m < kMT; ++m) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t byte = h ? hi[m] : lo[m];
            sat[m][h] = byte & ~3u;
            shift[m][h] = (byte & 3u) * 8;
            sw[m][h] = lds32(sat[m][h]);
        }
        if (!kSome || nb > 0) load(next[m], 0, m);
    }
#pragma unroll
    for (int i = 0; i < kNB; i += 2) {
        if (kSome && i >= nb) break;
        uint32_t w[kMT][4];
        float wsc[kMT][2][2];   // scales of rows lane / 4 and 8 more, two blocks each
#pragma unroll
        for (int m = 0; m < kMT; ++m) {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[m][j] = next[m][j];
            if (i + 2 < kNB && (!kSome || i + 2 < nb)) load(next[m], i + 2, m);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (i % 4 == 0) {   // the scales of four blocks, shifted into place
                    const uint32_t up = lds32(sat[m][h] + i + 4);
                    sc[m][h] = __funnelshift_r(sw[m][h], up, shift[m][h]);
                    if (kSome && nb - i < 4) sc[m][h] &= (1u << 8 * (nb - i)) - 1;
                    sw[m][h] = up;
                }
                scale_pair(sc[m][h], i % 4 != 0, wsc[m][h][0], wsc[m][h][1]);
            }
        }
#pragma unroll
        for (int h = 0; h < 2 && i + h < kNB; ++h) {
            const float2 x = *reinterpret_cast<const float2*>(sx + (i + h) * kCols);
#pragma unroll
            for (int m = 0; m < kMT; ++m) {
                uint32_t p[4], q[4];
                codes_to_f16(w[m][2 * h], p);
                codes_to_f16(w[m][2 * h + 1], q);
                float d[4];
                mma_f16_first(d, p[0], q[0], p[1], q[1], B[i + h][0], B[i + h][1]);
                mma_f16(d, p[2], q[2], p[3], q[3], B[i + h][2], B[i + h][3]);
#pragma unroll
                for (int t = 4; t < 4 * kTerms; t += 2) mma_f16(d, p[t - 4], q[t - 4], p[t - 3], q[t - 3], B[i + h][t], B[i + h][t + 1]);
                const float2 u = mul2(d[0], d[1], x), v = mul2(d[2], d[3], x);
                acc[m][0] = fmaf(u.x, wsc[m][0][h], acc[m][0]);
                acc[m][1] = fmaf(u.y, wsc[m][0][h], acc[m][1]);
                acc[m][2] = fmaf(v.x, wsc[m][1][h], acc[m][2]);
                acc[m][3] = fmaf(v.y, wsc[m][1][h], acc[m][3]);
            }
        }
    }
}

template <int kNB, int kMT, bool kBoxed, int kX, int kMode>
__global__ void __launch_bounds__(kThreads, 1) k_stream(const __grid_constant__ StreamArgs a) {
    using S = Shape<kNB, kMT, kBoxed>;
    constexpr bool kBoxes = S::kBoxes;
    constexpr bool kRoutes = kMode == kGlu || kMode == kDown;
    constexpr int kTerms = terms_of(kMode);
    extern __shared__ __align__(128) char sm[];
    __shared__ int scratch[kThreads / 32];
    uint64_t* full = reinterpret_cast<uint64_t*>(sm);   // a unit's copies have landed
    uint64_t* empty = full + kMaxStages;                // its consumers have read it
    uint64_t* done = empty + kMaxStages;                // [2 groups]: they have written their shares of the sums
    uint64_t* freed = done + 2 * kWarps;                // [2 groups]: the sums are formed
    float* red = reinterpret_cast<float*>(sm + S::kBars);
    float* sx_all = red + S::kRed / 4;
    int* seg = reinterpret_cast<int*>(sx_all + S::kSx / 4);
    int* first = seg + a.E + 1;
    uint16_t* list = reinterpret_cast<uint16_t*>(reinterpret_cast<char*>(seg) + (((a.E + 1) * 8 + 15) & ~15));
    char* ring = reinterpret_cast<char*>(list) + (kRoutes ? a.R * 2 : 0);
    ring += -tc::smem_u32(ring) & 1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long lim = a.wait_limit > 0 ? a.wait_limit : kDefaultWait;
    if (kRoutes) pdl_trigger();   // the next kernel may set itself up meanwhile
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            tc::mbar_init(full + s, 1);
            tc::mbar_init(empty + s, a.splits);
        }
        for (int i = 0; i < 2 * kWarps; ++i) {
            tc::mbar_init(done + i, a.splits);
            tc::mbar_init(freed + i, 1);
        }
        tc::fence_mbar_init();
    }
    group_rows<kMode>(a, seg, first, list, reinterpret_cast<int*>(ring), scratch);   // with barriers for the whole CTA
    // A stage holds kST tiles: boxes of [16 kST][128] swizzled bytes of codes, or rows, then scales; kGlu: 8 kST rows
    // of gate, then as many of up, in codes and scales alike.  A unit lies in kMT / kST stages one after the other.
    constexpr int kST = S::kStaged, kStages = kMT / kST;
    const int depth = a.K >> 5;                               // blocks of a weight row
    constexpr int rows_tile = kMode == kGlu ? 8 : 16;                                // features of a tile
    constexpr int features = rows_tile * kMT, staged = rows_tile * kST;              // of a unit, of a stage
    const int groups = a.groups;
    constexpr int box_bytes = 16 * kST * 128;
    const int code_bytes = kBoxes ? (a.slab_blocks + kBox - 1) / kBox * box_bytes : 16 * a.pitch;
    // scales of the second half of a tile are this far behind the first's
    const int half_bytes = kMode == kGlu ? (staged * a.scale_pitch + 31) & ~15 : 8 * a.scale_pitch;
    bool ok = true;               // no wait of this warp has expired
    int s = 0, ph = 0;
    Units it;
    it.start(first, a.E, (a.N + features - 1) / features, a.slabs);

    if (warp >= kWarps && warp < kWarps + 2) {
        // ---- producers: stages in turn ----
        const int me = warp - kWarps;
        const long long last = ((long long)a.E * a.N * depth) & ~15LL;   // the end of the scales' last whole piece of 16 bytes
        const int jobs = a.rows ? 16 : kMode == kGlu ? 2 : 1;            // runs of scales
        const long long total = (it.end - it.u) * kStages;
        constexpr int step = 2 / kStages;                                // units
        const int m = me % kStages;
        int n = me;                                                      // fill
        if (step == 2 && me) it.next(first);
        s = me % a.stages;
        for (; it.u < it.end; it.next(first, step), n += 2) {
            if (n >= a.stages && ok && !tc::mbar_wait(empty + s, ph ^ 1, lim)) ok = false;
            if (!__all_sync(0xffffffffu, ok)) break;
            const uint32_t to = s * a.stage_bytes;
            uint64_t* bar = full + s;
            if ((s += 2) >= a.stages) s -= a.stages, ph ^= 1;
            if (a.stall && n == 0) continue;   // test hook: the first stage never fills
            const int blk0 = it.slab * a.slab_blocks, nblk = min(a.slab_blocks, depth - blk0), boxes = (nblk + kBox - 1) / kBox;
            const int f0 = it.tile * features + m * staged, row0 = it.g * a.N + f0, rows = min(staged, a.N - f0);
            if (rows <= 0) {                   // a unit's second tile, past the last feature
                if (lane == 0) tc::mbar_arrive(bar);
                continue;
            }
            // Scales start anywhere, so the 16-byte pieces that hold them are copied, except behind the
            // tensor's last whole piece, where bytes go one by one.  Run j: `n` scales from `at` of their
            // tensor on, to the piece at `dst`.
            auto run = [&](int j, long long& at, int& count, uint32_t& dst, const uint8_t*& from) {
                const int half = kMode == kGlu ? (a.rows ? j / 8 : j) : 0, i = a.rows ? j - half * 8 : 0;
                at = (long long)(row0 + i) * depth + blk0;
                count = i >= rows ? 0 : a.rows ? nblk : rows * depth;
                dst = tc::smem_u32(ring) + to + code_bytes + half * half_bytes + i * a.scale_pitch;
                from = half ? a.scales2 : a.scales;
            };
            long long at;
            int count;
            uint32_t dst, bytes = 0;
            const uint8_t* from;
            for (int j = lane; j < jobs; j += 32) {
                run(j, at, count, dst, from);
                if (!count) continue;
                const long long piece = at & ~15LL;
                bytes += (uint32_t)(min((at + count + 15) & ~15LL, last) - piece);
                if (at + count > last) {
                    for (long long k = max(at, last); k < at + count; ++k)
                        asm volatile("st.shared.u8 [%0], %1;" ::"r"(dst + (uint32_t)(k - piece)), "r"((uint32_t)from[k]) : "memory");
                    tc::fence_proxy_async_smem();   // before a later unit's copy to the same place
                }
            }
            bytes = __reduce_add_sync(0xffffffffu, bytes) + (kBoxes ? boxes * box_bytes : rows * nblk * (kMode == kGlu ? 32 : 16));
            __syncwarp();   // the other lanes' bytes come before lane 0's arrival (a reduction orders no memory)
            if (lane == 0) {
                tc::mbar_expect_tx(bar, bytes);
                for (int b = 0; kBoxes && b < boxes; ++b) {
                    const int x = (blk0 + b * kBox) * 16;
                    tc::tma_load_2d(ring + to + b * box_bytes, &a.codes, bar, x, row0);
                    if (kMode == kGlu) tc::tma_load_2d(ring + to + b * box_bytes + box_bytes / 2, &a.codes2, bar, x, row0);
                }
            }
            __syncwarp();
            if (!kBoxes) {
                const int half = kMode == kGlu && lane >= 8, i = lane - half * 8;
                if (lane < 16 && i < rows) {
                        bulk_load(tc::smem_u32(ring) + to + lane * a.pitch, (half ? a.w2 : a.w) + ((long long)(row0 + i) * depth + blk0) * 16, nblk * 16, bar);
                }
            }
            for (int j = lane; j < jobs; j += 32) {
                run(j, at, count, dst, from);
                const long long piece = at & ~15LL;
                const uint32_t len = count ? (uint32_t)(min((at + count + 15) & ~15LL, last) - piece) : 0;
                if (len) bulk_load(dst, from + piece, len, bar);
            }
        }
        ok = __all_sync(0xffffffffu, ok);
        // No copy may be in flight when the CTA ends, also when the consumers gave up: the last fills of
        // each stage have landed.  (Fill n is the n / stages-th of stage n % stages.)
        for (int j = n - 2; j >= 0 && j > n - 2 - a.stages; j -= 2)
            if (!ok || j + a.stages >= total)
                if (!tc::mbar_wait(full + j % a.stages, (j / a.stages) & 1, ok ? lim : min(lim, 1LL << 10))) ok = false;
    } else if (warp >= kWarps) {
        // ---- sums of the consumers' shares, in order, a unit in turn.  Output o of a unit is column
        // o / 16 % kCols of tile o / (16 kCols), its row o % 16 or, for kGlu, such that neighbours hold
        // a feature's gate and up (rows 0 to 7 and 8 to 15 of a tile).
        const int me = warp - kWarps - 2;
        const int i = kMode == kGlu ? (lane & 1) << 3 | (lane >> 1 & 7) : lane & 15;
        int row0 = 0, nrows = 0, group = me % groups, turn = me / groups;
        if (me) it.next(first), it.fresh = true;
        for (; it.u < it.end; it.next(first, 2)) {
            if (it.fresh) {
                row0 = seg[it.g] + (it.chunk - first[it.g]) * kCols;
                nrows = min(kCols, seg[it.g + 1] - row0);
            }
            const int slot = 2 * group + (turn & 1);
            if (!tc::mbar_wait(done + slot, (turn >> 1) & 1, lim)) ok = false;
            if (!__all_sync(0xffffffffu, ok)) break;
            for (group += 2; group >= groups; group -= groups) ++turn;
            const float* base = red + slot * a.splits * (kMT * S::kPart) + i;
            for (int o = lane; o >> 5 < kMT * ((nrows + 1) >> 1); o += 32) {   // two columns at once, of those that exist
                const int pair = o >> 5, tile = kMT == 1 ? 0 : pair >= (nrows + 1) >> 1, c = 2 * (pair - tile * ((nrows + 1) >> 1)) + (lane >> 4);
                const float* p = base + tile * a.splits * S::kPart + c * kLine;
                float v[kWarps];
#pragma unroll
                for (int w = 0; w < kWarps; ++w) v[w] = w < a.splits ? p[w * S::kPart] : 0.0f;
#pragma unroll
                for (int w = 1; w < kWarps; ++w) v[0] += v[w];
                if (kMode == kGlu) {
                    const float u = __shfl_xor_sync(0xffffffffu, v[0], 1);
                    const int f = it.tile * features + tile * rows_tile + (i & 7);
                    if (c >= nrows || f >= a.N) continue;
                    const long long r = list[row0 + c];
                    float* y = static_cast<float*>(a.y);
                    if (a.slabs > 1) y[((it.slab * 2LL + (i >> 3)) * a.R + r) * a.ldy + f] = v[0];
                    else if (i < 8) y[r * a.ldy + f] = situ_glu(v[0], u, a.beta1, a.beta2);
                } else {
                    const int f = it.tile * features + tile * rows_tile + i;
                    if (c >= nrows || f >= a.N) continue;
                    const long long r = (kMode == kDown ? (int)list[row0 + c] : row0 + c) + (long long)it.slab * a.R;
                    if (kMode == kDown || a.y_type == QBMOE_F32) static_cast<float*>(a.y)[r * a.ldy + f] = v[0];
                    else static_cast<__nv_bfloat16*>(a.y)[r * a.ldy + f] = __float2bfloat16_rn(v[0]);
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(freed + slot);
        }
    } else {
        // ---- consumers ----
        const int group = warp / a.splits, wk = warp - group * a.splits;
        const int g8 = lane >> 2, t4 = lane & 3;
        float* sx = sx_all + warp * (kNB * kCols);
        if (kMode == kDown) pdl_wait();   // the rows come from the kernel before
        uint32_t B[kNB][4 * kTerms];
        int nb = 0, turn = 0;
        uint32_t wat0[4], sat0 = 0, start = 0;   // in stage 0: this lane's codes and scales; the first scale's place in its tensor
        const uint32_t in_second = a.rows && kMode != kGlu ? 8 * depth : 0;   // (row by row the second half's are elsewhere)
        float* mine0 = red + (2 * group * kMT * a.splits + wk) * S::kPart + 2 * t4 * kLine + g8;
        if (group) it.next(first, group), it.fresh = true;
        s = group * kStages;
        for (; it.u < it.end; it.next(first, groups), ++turn) {
            if (it.fresh) {
                const int blk0 = it.slab * a.slab_blocks, nblk = min(a.slab_blocks, depth - blk0);
                const int row0 = seg[it.g] + (it.chunk - first[it.g]) * kCols, nrows = min(kCols, seg[it.g + 1] - row0);
                const int per = kBoxes ? kNB : (nblk + a.splits - 1) / a.splits;
                const int b0 = wk * per;
                nb = max(0, min(per, nblk - b0));
                __syncwarp();
                const bool have = g8 < nrows;
                long long row = row0 + g8;
                if (kRoutes) row = have ? list[row0 + g8] : 0;
                if (kMode == kGlu) row = (int)row / a.k;
                // all loads of a batch before the first is used; blocks past the warp's share are zeros
                constexpr int kMost = kX == QBMOE_F32 ? 4 : 8, kBatch = kNB < kMost ? kNB : kMost;
#pragma unroll
                for (int i0 = 0; i0 < kNB; i0 += kBatch) {
                    Raw<kX> raw[kBatch];
#pragma unroll
                    for (int i = 0; i < kBatch && i0 + i < kNB; ++i) raw[i].load(a, row, blk0 + b0 + i0 + i, have && i0 + i < nb);
#pragma unroll
                    for (int i = 0; i < kBatch && i0 + i < kNB; ++i) {
                        const float sc = raw[i].template convert<kTerms>(B[i0 + i]);
                        if (t4 == 0) sx[(i0 + i) * kCols + g8] = sc;
                    }
                }
                __syncwarp();
                // ldmatrix: lanes 8 q .. 8 q + 7 give the rows of matrix q: rows 0 to 7 or 8 to 15 of block 0 or 1
                const int q = lane >> 3, half = q & 1, r = (kMode == kGlu ? staged : 8) * half + (lane & 7);
#pragma unroll
                for (int p = 0; p < (kBoxes ? 4 : 1); ++p) {
                    const int b = b0 + 2 * p + (q >> 1);
                    wat0[p] = tc::smem_u32(ring) + (kBoxes ? b0 / kBox * box_bytes + r * 128 + (((b & (kBox - 1)) ^ (r & 7)) << 4) : r * a.pitch + b * 16);
                }
                sat0 = tc::smem_u32(ring) + code_bytes + g8 * a.scale_pitch + b0;
                // scales start at a byte of their first 16: the unit's, or row by row each row's (then a unit is one tile)
                start = ((uint32_t)it.g * (uint32_t)a.N + (uint32_t)(it.tile * features + (a.rows ? g8 : 0))) * (uint32_t)depth + (uint32_t)blk0;
            }
            uint32_t at[kMT], lo[kMT], hi[kMT];
#pragma unroll
            for (int m = 0; m < kMT; ++m) {
                const bool wrap = s + m / kST >= a.stages;   // (one group: else its stages do not cross the ring's end)
                const int of = s + m / kST - (wrap ? a.stages : 0);
                // after a wait has expired nothing is waited for any more: what follows is undefined, and ends
                if (m % kST == 0 && ok && !tc::mbar_wait_spin(full + of, ph ^ (wrap ? 1 : 0), lim)) ok = false;
                const uint32_t stage = of * a.stage_bytes, in = m / kST * staged * depth, row = m % kST * rows_tile;
                at[m] = stage + row * 128;   // (rows one by one: a tile a stage)
                lo[m] = sat0 + stage + row * a.scale_pitch + ((start + in) & 15u);
                hi[m] = sat0 + stage + row * a.scale_pitch + half_bytes + ((start + in + in_second) & 15u);
            }
            start += groups * features * depth;
            float acc[kMT][4] = {};
            if (nb == kNB) share<kNB, kMT, kBoxes, false, kTerms>(B, sx + 2 * t4, wat0, at, lo, hi, nb, acc);
            else share<kNB, kMT, kBoxes, true, kTerms>(B, sx + 2 * t4, wat0, at, lo, hi, nb, acc);
            __syncwarp();
#pragma unroll
            for (int m = 0; m < kStages; ++m)
                if (lane == 0) tc::mbar_arrive(empty + (s + m >= a.stages ? s + m - a.stages : s + m));
            if ((s += groups * kStages) >= a.stages) s -= a.stages, ph ^= 1;
            const int slot = 2 * group + (turn & 1);
            if (ok && !tc::mbar_wait_spin(freed + slot, ((turn >> 1) & 1) ^ 1, lim)) ok = false;
#pragma unroll
            for (int m = 0; m < kMT; ++m) {
                float* mine = mine0 + ((turn & 1) * kMT + m) * a.splits * S::kPart;
                mine[0] = acc[m][0];
                mine[kLine] = acc[m][1];
                mine[8] = acc[m][2];
                mine[kLine + 8] = acc[m][3];
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(done + slot);
        }
    }
    if (!__all_sync(0xffffffffu, ok) && lane == 0 && a.expiries) atomicAdd(a.expiries, 1);
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
constexpr int kSlabBlocks = 256;   // of 32: the deepest slab that eight warps hold in 32 blocks each, or 16 of two terms

int slabs_of(int K, int mode = kStore) {
    const int most = kSlabBlocks / terms_of(mode);
    return (K / 32 + most - 1) / most;
}

// Calls f with the shape whose warps hold `per` blocks: the smallest of a few sizes (a warp with fewer leaves its loop
// after its last pair of blocks; a block missing from that pair is multiplied as zeros).  14 and 28 are K = 7 2^n; two
// tiles a unit halve what a unit costs besides, where the registers allow them.
template <int kMode, typename F>
int for_shape(bool boxes, int per, F f) {
    if constexpr (terms_of(kMode) == 2) {
        return boxes ? f(Shape<kBox, 2, true>{}) : f(Shape<16, 1, false>{});
    } else {
        if (boxes) return per <= kBox ? f(Shape<kBox, 2, true>{}) : f(Shape<2 * kBox, 2, true>{});
        if (per <= 14) return f(Shape<14, 2, false>{});
        if (per <= 16) return f(Shape<16, 2, false>{});
        if (per <= 28) return f(Shape<28, 1, false>{});
        return f(Shape<32, 1, false>{});
    }
}

// Geometry and launch; codes (kGlu: gate) and codes2 (up) are the weights' [E, N, K / 2].
template <int kX, int kMode>
int stream(StreamArgs a, const uint8_t* codes, const uint8_t* codes2, cudaStream_t s) {
    const int depth = a.K / 32;
    a.slabs = slabs_of(a.K, kMode);
    a.slab_blocks = ((depth + a.slabs - 1) / a.slabs + kBox - 1) / kBox * kBox;   // whole boxes
    a.slab_blocks = min(a.slab_blocks, depth);
    // short rows (up to eight boxes): the smallest groups whose warps have two each (of two terms, one); else all warps are one group
    const int n_boxes = (a.slab_blocks + kBox - 1) / kBox;
    const bool boxes = n_boxes <= 8;
    const int warp_boxes = n_boxes == 1 || terms_of(kMode) == 2 ? 1 : 2, holders = (n_boxes + warp_boxes - 1) / warp_boxes;
    a.splits = !boxes || holders > 4 ? kWarps : holders > 2 ? 4 : holders;
    a.groups = kWarps / a.splits;
    const int per = boxes ? warp_boxes * kBox : (a.slab_blocks + a.splits - 1) / a.splits;
    a.rows = a.slabs > 1;
    // row by row: pieces that hold a slab's scales from any start within 16 bytes, an odd number of
    // 16 bytes apart, so that eight rows lie in different banks
    a.scale_pitch = a.rows ? (((a.slab_blocks + 30) / 16) | 1) * 16 : depth;
    a.expiries = qbh::mx_expiries();
    a.wait_limit = qbh::mx_wait_limit();
    a.stall = qbh::mx_stall();
    return for_shape<kMode>(boxes, per, [&](auto shape) -> int {
        using S = decltype(shape);
        const int rows = 16 * S::kTiles, staged = 16 * S::kStaged, box_rows = kMode == kGlu ? staged / 2 : staged;
        a.w = codes;
        a.w2 = codes2;
        // long rows come one by one, an odd number of 16 bytes apart (ldmatrix without bank conflicts); short ones in boxes
        a.pitch = S::kBoxes ? 0 : (a.slab_blocks | 1) * 16;
        for (int i = 0; S::kBoxes && i < (codes2 ? 2 : 1); ++i)
            if (!qbh::encode_rows(i ? &a.codes2 : &a.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, i ? codes2 : codes, (long long)a.E * a.N, a.K / 2, a.K / 2,
                                  16 * kBox, box_rows))
                return QBMOE_ECUDA;
        const size_t code_bytes = a.pitch ? (size_t)16 * a.pitch : (size_t)(a.slab_blocks + kBox - 1) / kBox * staged * 128;
        a.stage_bytes = (int)qbh::align_up(code_bytes + staged * a.scale_pitch + 64, 1024);
        const size_t fixed = S::fixed(a.E, kMode == kStore ? 0 : a.R);
        a.stages = (int)((kMaxDynamic - kSlack - fixed) / a.stage_bytes);
        if (a.stages > kMaxStages) a.stages = kMaxStages;
        // Where groups take turns (2, 4 or 8 of them) a stage belongs to one of them, and to one producer:
        // a warp that waits for a barrier's next phase has then seen the one before, which a parity
        // cannot tell from the one after.
        if (a.groups > 1) a.stages -= a.stages % (a.groups * S::kTiles / S::kStaged);
        const size_t smem = fixed + (size_t)a.stages * a.stage_bytes + kSlack;   // two stages or more, and over the 32 KB that hist takes
        long long units = 0x7fffffff;
        if (kMode == kStore && !a.offsets) units = (((long long)a.R + kCols - 1) / kCols) * ((a.N + rows - 1) / rows) * a.slabs;
        const int grid = (int)min(units, (long long)qbh::sm_count());
        const auto kern = k_stream<S::kBlocks, S::kTiles, S::kBoxes, kX, kMode>;
        if (kMode == kDown) return qbh::launch_pdl(kern, dim3(grid), dim3(kThreads), smem, s, a);
        kern<<<grid, kThreads, smem, s>>>(a);
        return qbh::cuda_err(cudaGetLastError());
    });
}

template <int kX, int kMode>
int set_smem_all() {
    auto set = [](auto shape) {
        using S = decltype(shape);
        return qbh::cuda_err(cudaFuncSetAttribute(k_stream<S::kBlocks, S::kTiles, S::kBoxes, kX, kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamic));
    };
    int rc = 0;
    for (int per : {kBox, 2 * kBox})
        if (!rc) rc = for_shape<kMode>(true, per, set);
    for (int per : {14, 16, 28, 32})
        if (!rc) rc = for_shape<kMode>(false, per, set);
    return rc;
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
