// MXFP4 weights with few rows, and the routed experts of a few tokens (C ABI:
// moe_mxfp4_matvec, moe_mxfp4_experts).
//
// [K3-width] 延伸解读 on deployment: routed-expert weights in MXFP4; Q&A SiTU-GLU and
// RMSNorm: the experts' activation and the norm of their weighted sum.
//
// One kernel streams weights through shared memory and multiplies them with a few rows
// that stay in registers.  A persistent CTA a SM takes a contiguous run of units; a unit is
// 8 / splits tiles of 16 weight rows over the whole depth (or one slab of it).  Two producer
// warps bring a unit's codes and scales by untiled bulk copies, a row each, several units
// ahead.  Eight consumer warps divide the tiles and the depth: a warp owns a run of kNB
// blocks of 32 of K, for which it holds the rows' elements as mma B operands, so that the
// rows cost no bandwidth while weights go by.  Per block of 32 and tile:
//   - ldmatrix hands each quad of lanes the 16 bytes of a weight row's block;
//   - codes become fp16 (exact) two at a time, with one conversion;
//   - two m16n8k16 products, weights as A (16 rows), 8 columns of x as B;
//   - the block's dot products, times the two scales, are added in fp32.
// Two more warps add the shares of the depth, in order, and store.
// Weight rows are the M operand of the small mma because a column costs nothing that way: up
// to 8 rows of x take as long as one.  tcgen05 would need its operands decoded in shared
// memory, or x as E4M3 pairs (the layer's way: bound by issue at few columns).
#include "mxfp4.cuh"
#include "mxfp4_decode.cuh"
#include "tc_ptx.cuh"

#include <cuda_fp16.h>

#include <initializer_list>
#include <type_traits>

namespace {

using namespace qb;

constexpr int kWarps = 8;                      // consumers: all columns fit 168 registers a thread
constexpr int kFinishWarps = 2, kCodesWarp = 10;   // the last, 11, brings scales
constexpr int kThreads = 384;
constexpr int kMaxStages = 16;
constexpr int kLine = 20;                      // floats a column of 16 results takes: stores without bank conflicts
constexpr long long kDefaultWait = 1LL << 17;  // polls (<= 20 us each) before a wait expires
constexpr int kMaxDynamic = 226 * 1024;       // of 227 KB, a little being static
constexpr int kSlack = 512;                    // loads ahead of a warp's last blocks stay in shared memory

// What a launch computes.
enum { kStore, kGlu, kDown };

struct StreamArgs {
    int R, E, N, K;              // rows of x, experts, weight rows (features of kGlu), depth
    int x_type;
    const void* x;               // kDown: fp32 [R, K]
    long long ldx;
    const uint8_t* x_scales;
    const uint8_t *codes, *scales;       // [E, N, K / 2], [E, N, K / 32]
    const uint8_t *codes2, *scales2;     // kGlu: up (codes: gate)
    const int32_t* offsets;      // kStore: [E + 1] or NULL
    const int32_t* idx;          // kGlu, kDown: routes [R]
    int k;                       // kGlu: routes a token
    int y_type;
    void* y;                     // [slabs, R, N]; kGlu: fp32 [R, N], in slabs fp32 [slabs, 2, R, N]; kDown: fp32
    long long ldy;
    float beta1, beta2;
    // geometry
    int splits, split_log;       // consumers along the depth (a power of two); kWarps / splits tiles a unit
    int slabs, slab_blocks;      // the depth in slabs of this many blocks of 32
    int stages, stage_bytes, pitch, scale_pitch;
    int* expiries;
    long long wait_limit;
    int stall;
};

template <int kNB, int kNG>
struct Shape {
    static constexpr int kBlocks = kNB, kGroups = kNG;
    static constexpr int kCols = 8 * kNG;                      // rows of x a unit takes
    static constexpr int kPart = kCols * kLine + 8;            // floats of a warp's partial results
    static constexpr int kRed = 2 * kWarps * kPart * 4;        // double buffered
    static constexpr int kSx = kWarps * kNB * kCols * 4;       // scales of x
    static constexpr int kBars = (2 * kMaxStages + 4) * 8;
    static size_t fixed(int E, int routes) {
        return kBars + kRed + kSx + qbh::align_up((size_t)(E + 1) * 8, 16) + qbh::align_up((size_t)routes * 2, 16);
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
// Two E8M0 bytes, byte i of each word, as fp32 (0xFF: NaN).
QB_DEV void scale_pair(uint32_t lo, uint32_t hi, int i, float& a, float& b) {
    const uint32_t both = __byte_perm(lo, hi, (uint32_t)i | (uint32_t)(4 + i) << 4);
    uint32_t h;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.bf16x2.ue8m0x2 %0, l;\n\t}" : "=r"(h) : "r"(both));
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
// into [2^15, 65504], so that a bf16 element is exact down to 2^-32 of it, and any element within
// 2^-40 of it.  A block with an infinity or a NaN keeps those alone, which decide the result.
QB_DEV float block_to_f16(const float (&v)[8], uint32_t m, uint32_t (&b)[4]) {
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
    // The four pairs of fp16 and (in every lane of the quad) the block's scale.
    QB_DEV float convert(uint32_t (&b)[4]) const {
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
        return block_to_f16(f, m, b);
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
template <int kMode, int kCols>
QB_DEV void group_rows(const StreamArgs& a, int* seg, int* first, uint16_t* list, int* hist, int* scratch) {
    if (kMode == kGlu || kMode == kDown) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const int warps = min(kThreads / 32, (a.R + 31) >> 5), per = ((a.R + warps - 1) / warps + 31) & ~31;
        for (int i = threadIdx.x; i < warps * a.E; i += kThreads) hist[i] = 0;
        __syncthreads();
        for (int r = warp * per + lane; r < min(a.R, (warp + 1) * per); r += 32) {
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
        for (int r0 = warp * per; r0 < min(a.R, (warp + 1) * per); r0 += 32) {
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
    QB_DEV void next(const int* first) {
        ++u;
        fresh = false;
        if (++tile < tiles || u >= end) return;
        tile = 0;
        fresh = true;
        if (++chunk == chunks) chunk = 0, ++slab, g = 0;
        while (first[g + 1] <= chunk) ++g;
    }
};

// A warp's share of a tile: 16 weight rows times kNB blocks of K.  wat: this lane's row of the four
// 8 x 16-byte matrices that one ldmatrix loads (two blocks of 16 rows); lo, hi: the scales of
// weight rows lane / 4 and 8 more.  kSome: only nb blocks are the warp's; for the rest B and the
// scales of x are zeros, and the weights' scales, whatever lies there, are cleared lest one be NaN.
template <int kNB, int kNG, bool kSome>
QB_DEV void share(const uint32_t (&B)[kNB][kNG][4], const float* sx, uint32_t wat, uint32_t lo, uint32_t hi, int nb,
                  float (&acc)[kNG][4]) {
    uint32_t sat[2] = {lo & ~3u, hi & ~3u}, shift[2] = {(lo & 3u) * 8, (hi & 3u) * 8}, sw[2], sc[2], next[4];
    sw[0] = lds32(sat[0]);
    sw[1] = lds32(sat[1]);
    ldmatrix4(next, wat);
#pragma unroll
    for (int i = 0; i < kNB; i += 2) {
        if (kSome && i >= nb) break;
        const uint32_t w[4] = {next[0], next[1], next[2], next[3]};
        if (i + 2 < kNB) ldmatrix4(next, wat + (i + 2) * 16);
        if (i % 4 == 0) {   // the scales of four blocks, shifted into place
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t up = lds32(sat[h] + i + 4);
                sc[h] = __funnelshift_r(sw[h], up, shift[h]);
                if (kSome && nb - i < 4) sc[h] &= (1u << 8 * (nb - i)) - 1;
                sw[h] = up;
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t p[4], q[4];
            codes_to_f16(w[2 * h], p);
            codes_to_f16(w[2 * h + 1], q);
            float s0, s1;
            scale_pair(sc[0], sc[1], (i + h) & 3, s0, s1);
#pragma unroll
            for (int j = 0; j < kNG; ++j) {
                float d[4];
                mma_f16_first(d, p[0], q[0], p[1], q[1], B[i + h][j][0], B[i + h][j][1]);
                mma_f16(d, p[2], q[2], p[3], q[3], B[i + h][j][2], B[i + h][j][3]);
                const float2 x = *reinterpret_cast<const float2*>(sx + (i + h) * (8 * kNG) + 8 * j);
                const float2 u = mul2(d[0], d[1], x), v = mul2(d[2], d[3], x);
                acc[j][0] = fmaf(u.x, s0, acc[j][0]);
                acc[j][1] = fmaf(u.y, s0, acc[j][1]);
                acc[j][2] = fmaf(v.x, s1, acc[j][2]);
                acc[j][3] = fmaf(v.y, s1, acc[j][3]);
            }
        }
    }
}

template <int kNB, int kNG, int kX, int kMode>
__global__ void __launch_bounds__(kThreads, 1) k_stream(const StreamArgs a) {
    using S = Shape<kNB, kNG>;
    constexpr int kCols = S::kCols;
    constexpr bool kRoutes = kMode == kGlu || kMode == kDown;
    extern __shared__ __align__(128) char sm[];
    __shared__ int scratch[kThreads / 32];
    uint64_t* full = reinterpret_cast<uint64_t*>(sm);   // a unit's copies have landed
    uint64_t* empty = full + kMaxStages;                // its consumers have read it
    uint64_t* done = empty + kMaxStages;                // [2]: they have written their shares of the sums
    uint64_t* freed = done + 2;                         // [2]: the sums are formed
    float* red = reinterpret_cast<float*>(sm + S::kBars);
    float* sx_all = red + S::kRed / 4;
    int* seg = reinterpret_cast<int*>(sx_all + S::kSx / 4);
    int* first = seg + a.E + 1;
    uint16_t* list = reinterpret_cast<uint16_t*>(reinterpret_cast<char*>(seg) + (((a.E + 1) * 8 + 15) & ~15));
    char* ring = reinterpret_cast<char*>(list) + (kRoutes ? (a.R * 2 + 15) & ~15 : 0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long lim = a.wait_limit > 0 ? a.wait_limit : kDefaultWait;
    if (kRoutes) pdl_trigger();   // the next kernel may set itself up meanwhile
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            tc::mbar_init(full + s, 2);
            tc::mbar_init(empty + s, kWarps);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(done + i, kWarps);
            tc::mbar_init(freed + i, kFinishWarps);
        }
        tc::fence_mbar_init();
    }
    group_rows<kMode, kCols>(a, seg, first, list, reinterpret_cast<int*>(ring), scratch);   // with barriers for the whole CTA
    const int depth = a.K >> 5;                               // blocks of a weight row
    const int tiles_unit = kWarps >> a.split_log, rows_unit = 16 * tiles_unit;
    const int tile_rows = kMode == kGlu ? 8 * tiles_unit : rows_unit;   // features a unit
    bool ok = true;               // no wait of this warp has expired
    int s = 0, ph = 0, buf = 0;
    Units it;
    it.start(first, a.E, (a.N + tile_rows - 1) / tile_rows, a.slabs);

    if (warp >= kCodesWarp) {
        // ---- producers: a lane a row.  Codes are blocks of 16 bytes.  A row's scales start anywhere, so
        // the 16-byte pieces that hold them are copied, except behind the tensor's last whole
        // piece, where bytes go one by one.
        const bool codes = warp == kCodesWarp;
        const long long all = (long long)a.E * a.N * depth, last = all & ~15LL;
        int units = 0;
        for (; it.u < it.end; it.next(first), ++units) {
            if (units >= a.stages && !tc::mbar_wait(empty + s, ph ^ 1, lim)) ok = false;
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            const int blk0 = it.slab * a.slab_blocks, nblk = min(a.slab_blocks, depth - blk0);
            const uint32_t stage = tc::smem_u32(ring) + s * a.stage_bytes + (codes ? 0 : rows_unit * a.pitch);
            uint32_t bytes = 0, len[4];
            const uint8_t* from[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {   // at most 128 rows a unit
                const int i = lane + 32 * j;
                const int f = kMode == kGlu ? (it.tile * tiles_unit + (i >> 4)) * 8 + (i & 7) : it.tile * rows_unit + i;
                const bool up = kMode == kGlu && (i & 8);
                len[j] = 0;
                if (i >= rows_unit || f >= a.N) continue;
                const long long at = ((long long)it.g * a.N + f) * depth + blk0;
                if (codes) {
                    from[j] = (up ? a.codes2 : a.codes) + at * 16;
                    len[j] = nblk * 16;
                } else {
                    const long long piece = at & ~15LL;
                    const uint8_t* src = up ? a.scales2 : a.scales;
                    from[j] = src + piece;
                    len[j] = (uint32_t)(min((at + nblk + 15) & ~15LL, last) - piece);
                    if (at + nblk > last) {
                        for (long long k = max(at, last); k < at + nblk; ++k)
                            asm volatile("st.shared.u8 [%0], %1;" ::"r"(stage + i * a.scale_pitch + (uint32_t)(k - piece)), "r"((uint32_t)src[k]) : "memory");
                        tc::fence_proxy_async_smem();   // before a later unit's copy to the same place
                    }
                }
                bytes += len[j];
            }
            bytes = __reduce_add_sync(0xffffffffu, bytes);
            if (a.stall && codes && units == 0) bytes = 0;   // test hook: the first unit never arrives
            else if (lane == 0) tc::mbar_expect_tx(full + s, bytes);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (bytes && len[j]) bulk_load(stage + (lane + 32 * j) * (codes ? a.pitch : a.scale_pitch), from[j], len[j], full + s);
            if (++s == a.stages) s = 0, ph ^= 1;
        }
        // no copy may be in flight when the CTA ends, also after a wait has expired
        for (int i = 0; i < min(units, a.stages); ++i) {
            if (--s < 0) s = a.stages - 1, ph ^= 1;
            tc::mbar_wait(full + s, ph, ok ? lim : min(lim, 1LL << 10));
        }
    } else if (warp >= kWarps) {
        // ---- sums of the consumers' shares, in order.  Output o of a unit is column o / 16 % kCols of
        // tile o / (16 kCols), its row o % 16 or, for kGlu, such that neighbours hold a feature's gate
        // and up (rows 0 to 7 and 8 to 15 of a tile).
        constexpr int kLanes = 32 * kFinishWarps;
        const int o0 = threadIdx.x - 32 * kWarps;
        const int i = kMode == kGlu ? (o0 & 1) << 3 | (o0 >> 1 & 7) : o0 & 15;
        const int outputs = tiles_unit * 16 * kCols;
        int row0 = 0, nrows = 0;
        for (; it.u < it.end; it.next(first)) {
            if (it.fresh) {
                row0 = seg[it.g] + (it.chunk - first[it.g]) * kCols;
                nrows = min(kCols, seg[it.g + 1] - row0);
            }
            if (!tc::mbar_wait_spin(done + buf, ph, lim)) ok = false;
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            const float* from = red + buf * (kWarps * S::kPart) + i;
            for (int o = o0; o < outputs; o += kLanes) {
                const int c = (o >> 4) & (kCols - 1), tile = o / (16 * kCols);
                const float* p = from + (tile << a.split_log) * S::kPart + c * kLine;
                float v[kWarps];
#pragma unroll
                for (int w = 0; w < kWarps; ++w) v[w] = w < a.splits ? p[w * S::kPart] : 0.0f;
#pragma unroll
                for (int w = 1; w < kWarps; ++w) v[0] += v[w];
                if (kMode == kGlu) {
                    const float u = __shfl_xor_sync(0xffffffffu, v[0], 1);
                    const int f = (it.tile * tiles_unit + tile) * 8 + (i & 7);
                    if (c >= nrows || f >= a.N) continue;
                    const long long r = list[row0 + c];
                    float* y = static_cast<float*>(a.y);
                    if (a.slabs > 1) y[((it.slab * 2LL + (i >> 3)) * a.R + r) * a.ldy + f] = v[0];
                    else if (i < 8) y[r * a.ldy + f] = situ_glu(v[0], u, a.beta1, a.beta2);
                } else {
                    const int f = it.tile * rows_unit + tile * 16 + i;
                    if (c >= nrows || f >= a.N) continue;
                    const long long r = (kMode == kDown ? (int)list[row0 + c] : row0 + c) + (long long)it.slab * a.R;
                    if (kMode == kDown || a.y_type == QBMOE_F32) static_cast<float*>(a.y)[r * a.ldy + f] = v[0];
                    else static_cast<__nv_bfloat16*>(a.y)[r * a.ldy + f] = __float2bfloat16_rn(v[0]);
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(freed + buf);
            if (buf ^= 1, !buf) ph ^= 1;
        }
    } else {
        // ---- consumers ----
        const int wm = warp >> a.split_log, wk = warp & (a.splits - 1);
        const int g8 = lane >> 2, t4 = lane & 3;
        float* sx = sx_all + warp * (kNB * kCols);
        if (kMode == kDown) pdl_wait();   // the rows come from the kernel before
        uint32_t B[kNB][kNG][4];
        int b0 = 0, nb = 0, fph = 0;
        uint32_t wat0 = 0, sat0 = 0, scale_at = 0;   // in stage 0: this lane's codes and scales; a row's first scale
        const uint32_t scale_8 = kMode == kGlu ? 0 : 8 * depth;
        for (; it.u < it.end; it.next(first)) {
            if (it.fresh) {
                const int blk0 = it.slab * a.slab_blocks, nblk = min(a.slab_blocks, depth - blk0);
                const int row0 = seg[it.g] + (it.chunk - first[it.g]) * kCols, nrows = min(kCols, seg[it.g + 1] - row0);
                const int per = ((nblk - 1) >> a.split_log) + 1;
                b0 = wk * per;
                nb = max(0, min(per, nblk - b0));
                __syncwarp();
#pragma unroll
                for (int j = 0; j < kNG; ++j) {
                    const int c = 8 * j + g8;
                    const bool have = c < nrows;
                    long long row = row0 + c;
                    if (kRoutes) row = have ? list[row0 + c] : 0;
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
                            const float sc = raw[i].convert(B[i0 + i][j]);
                            if (t4 == 0) sx[(i0 + i) * kCols + c] = sc;
                        }
                    }
                }
                __syncwarp();
                const int q = lane >> 3, i = wm * 16 + g8;
                wat0 = tc::smem_u32(ring) + (wm * 16 + (lane & 7) + (q & 1) * 8) * a.pitch + (b0 + (q >> 1)) * 16;
                sat0 = tc::smem_u32(ring) + rows_unit * a.pitch + i * a.scale_pitch + b0;
                const int f = kMode == kGlu ? (it.tile * tiles_unit + wm) * 8 + g8 : it.tile * rows_unit + i;
                scale_at = ((uint32_t)it.g * (uint32_t)a.N + (uint32_t)f) * (uint32_t)depth + (uint32_t)blk0;
            }
            if (!tc::mbar_wait_spin(full + s, ph, lim)) ok = false;
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            float acc[kNG][4] = {};
            const uint32_t wat = wat0 + s * a.stage_bytes, sat = sat0 + s * a.stage_bytes;
            // a row's scales start at a byte of their first 16
            const uint32_t lo = sat + (scale_at & 15u), hi = sat + 8 * a.scale_pitch + ((scale_at + scale_8) & 15u);
            scale_at += tile_rows * depth;
            if (nb == kNB) share<kNB, kNG, false>(B, sx + 2 * t4, wat, lo, hi, nb, acc);
            else share<kNB, kNG, true>(B, sx + 2 * t4, wat, lo, hi, nb, acc);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(empty + s);
            if (++s == a.stages) s = 0, ph ^= 1;
            if (!tc::mbar_wait_spin(freed + buf, fph ^ 1, lim)) ok = false;
            float* mine = red + (buf * kWarps + warp) * S::kPart;
#pragma unroll
            for (int j = 0; j < kNG; ++j) {
                mine[(8 * j + 2 * t4) * kLine + g8] = acc[j][0];
                mine[(8 * j + 2 * t4 + 1) * kLine + g8] = acc[j][1];
                mine[(8 * j + 2 * t4) * kLine + g8 + 8] = acc[j][2];
                mine[(8 * j + 2 * t4 + 1) * kLine + g8 + 8] = acc[j][3];
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(done + buf);
            if (buf ^= 1, !buf) fph ^= 1;
        }
    }
    if (!ok && lane == 0 && a.expiries) atomicAdd(a.expiries, 1);
}

// ---------------------------------------------------------------------------
// What is left after the stream: sums of slabs, and the combination.
// ---------------------------------------------------------------------------

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
constexpr int kCombineThreads = 256, kCombineKeep = 4;

// Four elements of a token's weighted sum, its routes in order.
QB_DEV float4 weighted(const CombineArgs& a, const int* e, const float* w, int t, int f) {
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = 0; i < a.k; ++i) {
        if (e[i] < 0 || e[i] >= a.E) continue;
        for (int b = 0; b < a.slabs; ++b) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(a.rows + (((long long)b * a.T + t) * a.k + i) * a.L + f));
            s.x = fmaf(w[i], v.x, s.x); s.y = fmaf(w[i], v.y, s.y); s.z = fmaf(w[i], v.z, s.z); s.w = fmaf(w[i], v.w, s.w);
        }
    }
    return s;
}

// A token a CTA: the weighted sum of its routes, and its norm.  Sums of up to
// kCombineKeep 4 kCombineThreads features stay in registers; wider ones are formed again.
__global__ void __launch_bounds__(kCombineThreads) k_combine(const CombineArgs a) {
    __shared__ float part[kCombineThreads / 32];
    __shared__ int e[QBMOE_MAX_TOPK];
    __shared__ float w[QBMOE_MAX_TOPK];
    const int t = blockIdx.x;
    if ((int)threadIdx.x < a.k) {
        e[threadIdx.x] = a.idx[(long long)t * a.k + threadIdx.x];
        w[threadIdx.x] = a.w[(long long)t * a.k + threadIdx.x];
    }
    __syncthreads();
    pdl_wait();
    const int n = a.L >> 2;
    float4 keep[kCombineKeep];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < kCombineKeep; ++i) {
        const int at = threadIdx.x + i * kCombineThreads;
        if (at < n) keep[i] = weighted(a, e, w, t, 4 * at);
    }
    auto square = [&](const float4& v) { ss = fmaf(v.x, v.x, fmaf(v.y, v.y, fmaf(v.z, v.z, fmaf(v.w, v.w, ss)))); };
#pragma unroll
    for (int i = 0; i < kCombineKeep; ++i)
        if ((int)threadIdx.x + i * kCombineThreads < n) square(keep[i]);
    for (int at = threadIdx.x + kCombineKeep * kCombineThreads; at < n; at += kCombineThreads) square(weighted(a, e, w, t, 4 * at));
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
    for (int at = threadIdx.x + kCombineKeep * kCombineThreads; at < n; at += kCombineThreads) store(at, weighted(a, e, w, t, 4 * at));
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
constexpr int kSlabBlocks = 32 * kWarps;   // of 32: the deepest slab that the warps hold

int slabs_of(int K) { return (K / 32 + kSlabBlocks - 1) / kSlabBlocks; }

// Calls f with the shape whose warps hold `per` blocks of ng groups of 8 rows: the smallest of a
// few sizes (what is beyond a warp's share is multiplied with zeros).  14 and 28 are K = 7 2^n.
template <typename F>
int for_shape(int ng, int per, F f) {
    if (ng == 2) {
        if (per <= 4) return f(Shape<4, 2>{});
        if (per <= 8) return f(Shape<8, 2>{});
        if (per <= 14) return f(Shape<14, 2>{});
        return f(Shape<16, 2>{});
    }
    if (per <= 4) return f(Shape<4, 1>{});
    if (per <= 8) return f(Shape<8, 1>{});
    if (per <= 14) return f(Shape<14, 1>{});
    if (per <= 16) return f(Shape<16, 1>{});
    if (per <= 28) return f(Shape<28, 1>{});
    return f(Shape<32, 1>{});
}

// Geometry and launch.  Two groups of columns where experts have more than 8 rows on average
// and the depth allows it.
template <int kX, int kMode>
int stream(StreamArgs a, cudaStream_t s) {
    const int depth = a.K / 32;
    const int ng = depth <= 16 * kWarps && (long long)a.R > 8LL * a.E ? 2 : 1;
    a.slabs = slabs_of(a.K);
    a.slab_blocks = (depth + a.slabs - 1) / a.slabs;
    a.pitch = (a.slab_blocks | 1) * 16;                         // odd in 16 bytes: ldmatrix without bank conflicts
    a.scale_pitch = (((a.slab_blocks + 30) / 16) | 1) * 16;     // from any start within 16 bytes
    // the fewest splits for which a warp's share is at most 16 blocks (a unit's fixed work then counts little) ..
    while ((kWarps >> a.split_log) > 1 && (a.slab_blocks - 1) >> a.split_log >= 16) ++a.split_log;
    a.splits = 1 << a.split_log;
    const int per = ((a.slab_blocks - 1) >> a.split_log) + 1;
    const int rows = 16 * (kWarps / a.splits);
    a.stage_bytes = rows * (a.pitch + a.scale_pitch);
    a.expiries = qbh::mx_expiries();
    a.wait_limit = qbh::mx_wait_limit();
    a.stall = qbh::mx_stall();
    return for_shape(ng, per, [&](auto shape) {
        using S = decltype(shape);
        const size_t fixed = S::fixed(a.E, kMode == kStore ? 0 : a.R);
        a.stages = (int)((kMaxDynamic - kSlack - fixed) / a.stage_bytes);
        if (a.stages > kMaxStages) a.stages = kMaxStages;
        const size_t smem = fixed + (size_t)a.stages * a.stage_bytes + kSlack;   // two stages or more, and over the 48 KB that hist takes
        const int unit = kMode == kGlu ? rows / 2 : rows;
        long long units = 0x7fffffff;
        if (kMode == kStore && !a.offsets) units = (((long long)a.R + S::kCols - 1) / S::kCols) * ((a.N + unit - 1) / unit) * a.slabs;
        const int grid = (int)min(units, (long long)qbh::sm_count());
        const auto kern = k_stream<S::kBlocks, S::kGroups, kX, kMode>;
        if (kMode == kDown) return qbh::launch_pdl(kern, dim3(grid), dim3(kThreads), smem, s, a);
        kern<<<grid, kThreads, smem, s>>>(a);
        return qbh::cuda_err(cudaGetLastError());
    });
}

template <int kNB, int kNG, int kX, int kMode>
int set_smem() {
    return qbh::cuda_err(cudaFuncSetAttribute(k_stream<kNB, kNG, kX, kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamic));
}
template <int kX, int kMode>
int set_smem_all() {
    int rc = 0;
    for (int ng = 1; ng <= 2; ++ng)
        for (int per : {4, 8, 14, 16, 28, 32})
            if (!rc && per <= 32 / ng)
                rc = for_shape(ng, per, [](auto shape) { return set_smem<decltype(shape)::kBlocks, decltype(shape)::kGroups, kX, kMode>(); });
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

// Scratch of an experts call: act; gate and up in slabs; the routes' rows.
struct ExpertsScratch {
    size_t act, parts, rows, bytes;
    ExpertsScratch(int T, int k, int L, int M) {
        const size_t R = (size_t)T * k, up = slabs_of(L), down = slabs_of(M);
        act = 0;
        parts = qbh::align_up(R * M * 4, 256);
        rows = parts + (up > 1 ? qbh::align_up(up * 2 * R * M * 4, 256) : 0);
        bytes = rows + qbh::align_up(down * R * L * 4, 256);
    }
};

}  // namespace

namespace qbh {

int matvec_init() {
    int rc = set_smem_all<QBMOE_BF16, kStore>();
    if (!rc) rc = set_smem_all<QBMOE_MXFP8, kStore>();
    if (!rc) rc = set_smem_all<QBMOE_BF16, kGlu>();
    if (!rc) rc = set_smem_all<QBMOE_MXFP8, kGlu>();
    if (!rc) rc = set_smem_all<QBMOE_F32, kDown>();
    return rc;
}

}  // namespace qbh

extern "C" size_t qbmoe_mxfp4_matvec_workspace_bytes(int R, int N, int K) {
    if (R < 0 || R > QBMOE_MAX_ROWS || N < 8 || N % 8 || N > kMaxCols || !depth_ok(K) || slabs_of(K) == 1) return 0;
    return (size_t)slabs_of(K) * R * N * 4;
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
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    StreamArgs a{};
    a.R = R; a.E = E; a.N = N; a.K = K;
    a.x_type = x_type; a.x = x; a.ldx = ldx; a.x_scales = x_scales;
    a.codes = w_codes; a.scales = w_scales; a.offsets = offsets;
    a.y_type = need ? QBMOE_F32 : y_type;
    a.y = need ? workspace : y;
    a.ldy = need ? N : ldy;
    const int rc2 = x_type == QBMOE_BF16 ? ::stream<QBMOE_BF16, kStore>(a, s) : ::stream<QBMOE_MXFP8, kStore>(a, s);
    if (rc2 || !need) return rc2;
    const long long blocks = ((long long)R * N + 255) / 256;
    k_slab_sum<<<(unsigned)min(blocks, 8LL * qbh::sm_count()), 256, 0, s>>>(slabs_of(K), R, N, E, offsets, static_cast<float*>(workspace), y_type, y, ldy);
    return qbh::cuda_err(cudaGetLastError());
}

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
    if (!(beta1 > 0.0f) || !(beta2 > 0.0f) || !(rms_eps >= 0.0f)) return QBMOE_EINVAL;
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
    StreamArgs a{};
    a.R = T * k; a.E = E; a.N = M; a.K = L;
    a.x_type = x_type; a.x = x; a.ldx = ldx; a.x_scales = x_scales;
    a.codes = gate_codes; a.scales = gate_scales; a.codes2 = up_codes; a.scales2 = up_scales;
    a.idx = idx; a.k = k;
    a.y_type = QBMOE_F32; a.y = slabs_of(L) > 1 ? parts : act; a.ldy = M;
    a.beta1 = beta1; a.beta2 = beta2;
    int rc2 = x_type == QBMOE_BF16 ? ::stream<QBMOE_BF16, kGlu>(a, s) : ::stream<QBMOE_MXFP8, kGlu>(a, s);
    if (rc2) return rc2;
    if (slabs_of(L) > 1) {
        const long long blocks = ((long long)a.R * M + 255) / 256;
        k_glu_sum<<<(unsigned)min(blocks, 8LL * qbh::sm_count()), 256, 0, s>>>(slabs_of(L), a.R, M, E, idx, parts, beta1, beta2, act);
        if ((rc2 = qbh::cuda_err(cudaGetLastError()))) return rc2;
    }
    StreamArgs d = a;
    d.N = L; d.K = M;
    d.x_type = QBMOE_F32; d.x = act; d.ldx = M; d.x_scales = nullptr;
    d.codes = out_codes; d.scales = out_scales; d.codes2 = d.scales2 = nullptr;
    d.y = rows; d.ldy = L;
    if ((rc2 = ::stream<QBMOE_F32, kDown>(d, s))) return rc2;
    const CombineArgs c{T, k, E, L, slabs_of(M), idx, w, rows, gamma, rms_eps, static_cast<__nv_bfloat16*>(y), ldy};
    return qbh::launch_pdl(k_combine, dim3(T), dim3(kCombineThreads), 0, s, c);
}
