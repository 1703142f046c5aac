// MXFP4 product y = x w^T on the block-scaled tensor cores of sm_103a.
//
// Mathematics: y[r][f] = sum_b 2^(ex[r][b] + ew[f][b]) sum_(k in b) cx[r][k] cw[f][k]
// over blocks b of 32 elements; tcgen05.mma kind::mxf4 takes the packed E2M1
// codes from shared memory as they lie in HBM and both operands' E8M0 scales
// from TMEM, and accumulates in fp32.
//
// Orientation: the weights are the MMA's A operand (M = 128 rows) and the
// expert's rows its B operand (N = 16 .. BN), so that a decode step with a few
// rows an expert still issues full-height MMAs while it streams the weights.
//
// One persistent warp-specialised kernel.  A stage is 256 elements of K: the
// packed codes of 128 weight rows and of the tile's rows (128 bytes each, TMA,
// 128-byte swizzle); their scales come in groups of two stages (16 bytes a row).
//   warp 0      TMA producer of the weights' codes (one lane); once it has a free
//               stage it meets the scale writers at a named barrier (a
//               suspended mbarrier wait takes about a microsecond to come back, and
//               every warp that polls instead slows the others)
//   last warp   TMA producer of the rows' codes (one lane that issued both took 570
//               cycles a stage)
//   warp 1      TMEM owner, MMA issuer (one elected lane; a branch on the lane number
//               makes the issue slower: 567 against 545 us at the prefill case): 4 x
//               K = 64 MMAs a stage and one commit that frees it
//   warp 2      the issuer's waiter (an mbarrier wait by the issuing thread
//               slows its MMA stream): waits, then releases it through a named barrier
//   warp 3      scale groups to shared memory: by TMA (one lane) where the scale
//               rows are multiples of 16 bytes (K % 512 == 0), else through
//               registers, a group ahead
//   warps 4-7   scale writers, one per TMEM lane quarter: a group's scales from
//               shared memory to the stages' TMEM slots (tcgen05.st).  Copying them
//               with tcgen05.cp from the issuer cost it 6 more instructions a
//               stage: 813 cycles of issue, against 375 of MMAs at N = 192.
//   warps 8+    epilogue, two warps per lane quarter (one on 16-row tiles): TMEM
//               -> bf16 pairs of features -> 64 bytes a row and warp
// Two accumulators alternate, so a tile's epilogue overlaps the next tile's
// main loop.
//
// Measured (weights 1024 x 3584 an expert): 4096 rows over 896 experts 252 us, the
// packed weights at 6.9 TB/s; 262144 rows over 896 experts 508 us (3.8 PFLOP/s, 5.5 TB/s);
// 1999 rows by 3584 x 7168 24 us (4.3 PFLOP/s).  16-row tiles are bound by HBM, larger
// ones by the time a stage's slot is held (copies and hand-offs, about 3000 cycles, of
// which the MMAs are 300 to 400): what fits in flight counts.  Tiles of 192 rows
// with five slots take 508 us where 208 with four take 545, 160 with five 538, 144 with
// six 532 and 128 with six 558 (with five 599).
// Scale rows that TMA cannot copy (K % 512 != 0) cost the loading warp one to sixteen
// loads a row and group.  16384 rows over 56 experts of 1024 x K: K = 3584 (TMA) 53 us,
// 3328 (8-byte loads) 65, 3456 (4-byte) 71, 3360 (1-byte) 378; one row by 6144 x K: 15.5,
// 15.5, 15.5 and 35 us.  The last is bound by those loads alone.
// Every mbarrier wait is bounded: on expiry the kernel counts it
// (mx_expiries), stops, lets its own copies and MMAs finish and frees TMEM.
#include "mxfp4.cuh"
#include "tc_ptx.cuh"

#include <cudaTypedefs.h>

#include <mutex>

namespace {

using namespace qb;

constexpr int kStageK = 256;                 // elements of K per stage (128 bytes of codes a row)
constexpr int kABytes = 128 * 128;           // weight codes of a stage
constexpr int kMmaWarp = 1, kWaitWarp = 2, kSfLoadWarp = 3, kSfWarp = 4, kEpiWarp = 8;
constexpr int kHandoffBar = 1, kEpiBar = 2, kStageBar = 3;
constexpr int kMaxBoxes = 4;                 // row-tile maps: heights BN / n, 2 BN / n, ...
constexpr long long kDefaultWait = 1LL << 17;   // polls (<= 20 us each) before a wait expires
constexpr long long kDrainWait = 1LL << 12;

struct Params {
    CUtensorMap a;                           // codes of the weights [E N, K / 2]
    CUtensorMap b[kMaxBoxes];                // and of the rows [R, K / 2], one map per box height
    CUtensorMap a_sf, b_sf;                  // their scales [., K / 32] (K % 512 == 0)
    const uint8_t* a_sc;
    const uint8_t* b_sc;
    const int32_t* offsets;
    __nv_bfloat16* y;
    long long ldy;
    int R, E, N, K, nkb, m_total;
    int sf_tma;                              // scale groups by TMA
    int sf_bytes;                            // else bytes of a scale load: 8 (K % 256 == 0), 4 (K % 128 == 0) or 1
    int weights_ready;                       // nothing enqueued just before this kernel wrote the weights or the offsets
    int* expiries;
    long long wait_limit;
    int stall;                               // test hook: withhold the first accumulator hand-off
};

template <int BN>
struct Shape {
    static constexpr int kEpiWarps = BN == 16 ? 4 : 8;
    static constexpr int kProdBWarp = kEpiWarp + kEpiWarps;
    static constexpr int kThreads = (kProdBWarp + 1) * 32;
    static constexpr int kBoxes = BN > 128 ? 4 : BN == 128 ? 2 : 1;
    static constexpr int kBox = BN / kBoxes;                     // a row tile is one copy, of the least multiple that holds it
    static constexpr int kNB = (BN + 127) / 128;                 // 128-row blocks of B's scales
    static constexpr int kBJ = (BN + 31) / 32;                   // 32-row blocks
    static constexpr int kBBytes = BN * 128;
    static constexpr int kStage = kABytes + kBBytes;
    static constexpr int kSfBytes = (128 + BN) * 16;             // scales of a group
    static constexpr int kSfCols = 8 + 8 * kNB;                  // TMEM columns of a stage's scales
    static constexpr int kSfSlots = BN <= 64 ? 4 : 3;            // scale groups in flight, of two stages each
    static constexpr int stages = BN == 64 ? 7 : BN == 128 ? 6 : BN == 192 ? 5 : 4;
    static constexpr int kColsUsed = 2 * BN + stages * kSfCols;  // two accumulators, a scale slot per stage
    static constexpr uint32_t kCols = kColsUsed <= 128 ? 128 : kColsUsed <= 256 ? 256 : 512;
    static_assert(kColsUsed <= 512, "TMEM columns");
    static_assert(stages <= 2 * kSfSlots, "scales in flight for every stage");
    static constexpr int smem(int E) {
        return 1024 + stages * kStage + kSfSlots * kSfBytes + (2 * (E + 1) + 64) * 4 + 256;
    }
};

// kind::mxf4 instruction descriptor: A and B E2M1 (format 1), K-major, E8M0
// scales (bit 23), M = 128, N = n; the scale ids (bits 4 and 29) pick the
// byte pair of the 32-bit scale words that this K = 64 slice uses (0 or 2).
__device__ __forceinline__ uint32_t idesc_mxf4(uint32_t n, uint32_t sf) {
    return (sf << 4) | (1u << 7) | (1u << 10) | ((n >> 3) << 17) | (1u << 23) | ((128u >> 4) << 24) | (sf << 29);
}
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
// 16 scale bytes of one row (a group of two stages); bytes past the row's end
// are 0 (their codes are, too).
__device__ __forceinline__ uint4 load_scales(const uint8_t* row, int pitch, int at, int bytes) {
    const uint8_t* p = row + at;
    const int left = pitch - at;
    uint32_t v[4] = {0, 0, 0, 0};
    if (bytes == 8) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
        v[0] = x.x, v[1] = x.y;
        if (left > 8) {
            const uint2 y = __ldg(reinterpret_cast<const uint2*>(p) + 1);
            v[2] = y.x, v[3] = y.y;
        }
    } else if (bytes == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (left > 4 * i) v[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (left > i) v[i >> 2] |= (uint32_t)__ldg(p + i) << (8 * (i & 3));
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

template <int BN>
__global__ void __launch_bounds__(Shape<BN>::kThreads, BN == 16 ? 2 : 1) k_mx_product(const __grid_constant__ Params p) {
    using Sh = Shape<BN>;
    constexpr int S = Sh::stages, kSfSlots = Sh::kSfSlots;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* a_ring = smem;
    uint8_t* b_ring = a_ring + S * kABytes;
    uint8_t* sf_ring = b_ring + S * Sh::kBBytes;                 // [kSfSlots][128 + BN rows][16]
    uint64_t* full = reinterpret_cast<uint64_t*>(sf_ring + kSfSlots * Sh::kSfBytes);
    uint64_t* empty = full + S;
    uint64_t* sf_full = empty + S;
    uint64_t* sf_empty = sf_full + kSfSlots;
    uint64_t* accf = sf_empty + kSfSlots;
    uint64_t* acce = accf + 2;
    uint64_t* drain = acce + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* go_flag = reinterpret_cast<volatile int*>(tmem_slot + 2);   // [2]
    int* scratch = reinterpret_cast<int*>(tmem_slot + 4);                     // [kThreads / 32]
    Groups gr;
    gr.seg = scratch + 24;
    gr.toff = gr.seg + p.E + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long lim = p.wait_limit > 0 ? p.wait_limit : kDefaultWait;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            tc::mbar_init(&full[s], 6);      // the two TMA producers and four scale writers
            tc::mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < kSfSlots; ++a) {
            tc::mbar_init(&sf_full[a], 1);
            tc::mbar_init(&sf_empty[a], 4);
        }
        for (int a = 0; a < 2; ++a) {
            tc::mbar_init(&accf[a], 1);
            tc::mbar_init(&acce[a], Sh::kEpiWarps);
        }
        tc::mbar_init(drain, 1);
        *abort_flag = 0;
        tc::fence_mbar_init();
        tc::fence_proxy_async_smem();
        tc::prefetch_tmap(&p.a);
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(tmem_slot, Sh::kCols);
        tc::tmem_relinquish();
    }
    if (!p.weights_ready) pdl_wait();
    tc::tc_fence_before();
    load_groups<BN, Sh::kThreads>(gr, p.offsets, p.E, p.R, scratch);
    tc::tc_fence_after();
    const uint32_t tbase = *tmem_slot;
    const int n_tiles = gr.toff[p.E] * p.m_total;
    Walker<BN> w;
    w.start(gr, p.E, p.m_total);
    const int first = blockIdx.x, step = gridDim.x;
    auto expired = [&] {
        if (p.expiries) atomicAdd(p.expiries, 1);
        *abort_flag = 1;
    };

    if (warp == 0 || warp == Sh::kProdBWarp) {
        // ---------------------------------------------------------- TMA producers
        const bool is_a = warp == 0;
        uint32_t issued = 0, last_par = 0;
        int s = 0;
        uint32_t ph = 0;
        if (!is_a && p.weights_ready) pdl_wait();   // the rows' codes come from the kernel before this one
        bool dead = false;   // lane 0: an expiry; only the meetings go on
        for (int t = first; t < n_tiles; t += step) {
            const int box = (w.nrows - 1) / Sh::kBox;
            const CUtensorMap* map = is_a ? &p.a : &p.b[box];
            const int row = is_a ? w.g * p.N + w.m * 128 : w.row0;
            const uint32_t bytes = is_a ? kABytes : (box + 1) * Sh::kBox * 128;
            constexpr int kAStride = kABytes, kBStride = Sh::kBBytes;
            const int stride = is_a ? kAStride : kBStride;
            uint8_t* ring = is_a ? a_ring : b_ring;
            w.next(gr, p.E, p.m_total);
            if (lane == 0 && *abort_flag) dead = true;
            for (int kb = 0; kb < p.nkb; ++kb) {
                if (lane == 0 && !dead && !tc::mbar_wait_spin(&empty[s], ph ^ 1u, lim)) { expired(); dead = true; }
                if (lane == 0 && !dead) {
                    tc::mbar_expect_tx(&full[s], bytes);
                    tc::tma_load_2d(ring + s * stride, map, &full[s], kb * 128, row);
                    issued |= 1u << s;
                    last_par = (last_par & ~(1u << s)) | (ph << s);
                }
                __syncwarp();
                if (is_a) tc::named_bar_sync(kStageBar, 160);
                if (++s == S) { s = 0; ph ^= 1u; }
            }
        }
        __syncthreads();
        if (lane == 0 && *abort_flag)   // every copy has landed before shared memory is released
            for (int i = 0; i < S; ++i)
                if ((issued >> i) & 1u) tc::mbar_wait(&full[i], (last_par >> i) & 1u, kDrainWait);
    } else if (warp == kSfLoadWarp) {
        // ---------------------------------------------------------- scale groups
        // Without TMA, lane l takes rows l, l + 32, ... of the weight tile and of
        // the row tile; the next group's bytes are in registers while it waits
        // for a slot.
        uint32_t sf_issued = 0, sf_par = 0;
        if (p.weights_ready) pdl_wait();
        if (p.sf_tma) {
            int gs = 0;
            uint32_t gph = 0;
            for (int t = first; t < n_tiles; t += step) {
                const int ya = w.g * p.N + w.m * 128, yb = w.row0;
                w.next(gr, p.E, p.m_total);
                int stop = 0;
                if (lane == 0) {
                    stop = *abort_flag;
                    for (int kb = 0; kb < p.nkb && !stop; kb += 2) {
                        if (!tc::mbar_wait_spin(&sf_empty[gs], gph ^ 1u, lim)) { expired(); stop = 1; break; }
                        uint8_t* SF = sf_ring + gs * Sh::kSfBytes;
                        tc::mbar_expect_tx(&sf_full[gs], Sh::kSfBytes);
                        tc::tma_load_2d(SF, &p.a_sf, &sf_full[gs], kb * 8, ya);
                        tc::tma_load_2d(SF + 128 * 16, &p.b_sf, &sf_full[gs], kb * 8, yb);
                        sf_issued |= 1u << gs;
                        sf_par = (sf_par & ~(1u << gs)) | (gph << gs);
                        if (++gs == kSfSlots) { gs = 0; gph ^= 1u; }
                    }
                }
                if (__shfl_sync(0xffffffffu, stop, 0)) break;
            }
        } else {
            const int pitch = p.K / 32;
            const long long last_a = (long long)p.E * p.N - 1;
            uint4 ra[4], rb[Sh::kBJ];
            auto fetch = [&](int kb) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const long long row = min((long long)w.g * p.N + w.m * 128 + lane + 32 * j, last_a);
                    ra[j] = load_scales(p.a_sc + row * pitch, pitch, kb * 8, p.sf_bytes);
                }
#pragma unroll
                for (int j = 0; j < Sh::kBJ; ++j) {
                    const int r = min(w.row0 + lane + 32 * j, p.R - 1);
                    rb[j] = 32 * j < w.nrows ? load_scales(p.b_sc + (long long)r * pitch, pitch, kb * 8, p.sf_bytes)
                                             : make_uint4(0, 0, 0, 0);
                }
            };
            int gs = 0, kb = 0, t = first;
            uint32_t gph = 0;
            if (t < n_tiles) fetch(0);
            while (t < n_tiles) {
                int ok = 1;
                if (lane == 0) {
                    ok = !*abort_flag;
                    if (ok && !tc::mbar_wait_spin(&sf_empty[gs], gph ^ 1u, lim)) { expired(); ok = 0; }
                }
                if (!__shfl_sync(0xffffffffu, ok, 0)) break;
                uint4* SF = reinterpret_cast<uint4*>(sf_ring + gs * Sh::kSfBytes);
#pragma unroll
                for (int j = 0; j < 4; ++j) SF[lane + 32 * j] = ra[j];
#pragma unroll
                for (int j = 0; j < Sh::kBJ; ++j)
                    if (lane + 32 * j < BN) SF[128 + lane + 32 * j] = rb[j];
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sf_full[gs]);
                if (++gs == kSfSlots) { gs = 0; gph ^= 1u; }
                kb += 2;
                if (kb >= p.nkb) {
                    kb = 0;
                    t += step;
                    if (t < n_tiles) w.next(gr, p.E, p.m_total);
                }
                if (t < n_tiles) fetch(kb);
            }
        }
        __syncthreads();
        if (lane == 0 && *abort_flag)
            for (int i = 0; i < kSfSlots; ++i)
                if ((sf_issued >> i) & 1u) tc::mbar_wait(&sf_full[i], (sf_par >> i) & 1u, kDrainWait);
    } else if (warp >= kSfWarp && warp < kEpiWarp) {
        // ---------------------------------------------------------- scale writers
        // The MMA reads the scale words of row r (four bytes: K = 128) from lane
        // r % 32, column r / 32 of a slot, in each lane quarter.
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        int s = 0, gs = 0;
        uint32_t gph = 0;
        bool dead = false;
        for (int t = first; t < n_tiles; t += step) {
            if (lane == 0 && *abort_flag) dead = true;
            for (int kb0 = 0; kb0 < p.nkb; kb0 += 2) {
                const int stages = min(2, p.nkb - kb0);
                if (lane == 0 && !dead && !tc::mbar_wait_spin(&sf_full[gs], gph, lim)) { expired(); dead = true; }
                __syncwarp();
                const uint4* SF = reinterpret_cast<const uint4*>(sf_ring + gs * Sh::kSfBytes);
                uint4 ra[4], rb[4 * Sh::kNB];
#pragma unroll
                for (int j = 0; j < 4; ++j) ra[j] = SF[lane + 32 * j];
#pragma unroll
                for (int j = 0; j < 4 * Sh::kNB; ++j)
                    rb[j] = lane + 32 * j < BN ? SF[128 + lane + 32 * j] : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (u >= stages) break;
                    uint32_t va[8], vb[8 * Sh::kNB];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) va[4 * c + j] = word(ra[j], 2 * u + c);
#pragma unroll
                        for (int j = 0; j < 4 * Sh::kNB; ++j) vb[4 * Sh::kNB * c + j] = word(rb[j], 2 * u + c);
                    }
                    tc::named_bar_sync(kStageBar, 160);   // the stage's slot is free
                    tc::tc_fence_after();
                    const int at = s + u < S ? s + u : s + u - S;
                    const uint32_t slot = tbase + lanes + 2 * BN + at * Sh::kSfCols;
                    tc::tmem_st8(slot, va);
                    if constexpr (Sh::kNB == 2) tc::tmem_st16(slot + 8, vb); else tc::tmem_st8(slot + 8, vb);
                    tc::tmem_wait_st();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&full[at]);
                }
                if (lane == 0) tc::mbar_arrive(&sf_empty[gs]);   // read before the stages' arrivals
                s += stages;
                if (s >= S) s -= S;
                if (++gs == kSfSlots) { gs = 0; gph ^= 1u; }
            }
        }
        __syncthreads();
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------- MMA issuer
        int s = 0, ab = 0, h = 0;
        const uint64_t a0 = tc::desc_sw128(tc::smem_u32(a_ring)), b0 = tc::desc_sw128(tc::smem_u32(b_ring));
        for (int t = first; t < n_tiles; t += step) {
            const uint32_t n_eff = (w.nrows + 15) & ~15;
            const uint32_t id0 = idesc_mxf4(n_eff, 0), id2 = idesc_mxf4(n_eff, 2);
            w.next(gr, p.E, p.m_total);
            tc::named_bar_sync(kHandoffBar, 64);   // the accumulator is free (or stop)
            const bool go = go_flag[h & 1] != 0;
            ++h;
            if (!go) break;
            const uint32_t d = tbase + ab * BN;
            for (int kb = 0; kb < p.nkb; ++kb) {
                // the stage's addresses, before the wait for it
                const uint32_t ca = tbase + 2 * BN + s * Sh::kSfCols, cb = ca + 8;
                const uint64_t ad = a0 + (uint64_t)(s * (kABytes >> 4)), bd = b0 + (uint64_t)(s * (Sh::kBBytes >> 4));
                const int left = p.K - kb * kStageK;
                tc::named_bar_sync(kHandoffBar, 64);   // stage s has landed
                if (tc::elect_one()) {
                    tc::tc_fence_after();
                    mma_mxf4(d, ad, bd, id0, ca, cb, kb != 0);
                    if (left > 192) {
                        mma_mxf4(d, ad + 2, bd + 2, id2, ca, cb, 1);
                        mma_mxf4(d, ad + 4, bd + 4, id0, ca + 4, cb + 4 * Sh::kNB, 1);
                        mma_mxf4(d, ad + 6, bd + 6, id2, ca + 4, cb + 4 * Sh::kNB, 1);
                    } else {
                        if (left > 64) mma_mxf4(d, ad + 2, bd + 2, id2, ca, cb, 1);
                        if (left > 128) mma_mxf4(d, ad + 4, bd + 4, id0, ca + 4, cb + 4 * Sh::kNB, 1);
                    }
                    tc::tc_commit(&empty[s]);
                }
                __syncwarp();
                if (++s == S) s = 0;
            }
            if (tc::elect_one() && !(p.stall && t == first)) tc::tc_commit(&accf[ab]);
            __syncwarp();
            ab ^= 1;
        }
        if (tc::elect_one()) {   // every MMA of this thread is done before TMEM is freed
            tc::tc_commit(drain);
            tc::mbar_wait(drain, 0, kDefaultWait);
        }
        __syncwarp();
        __syncthreads();
    } else if (warp == kWaitWarp) {
        // ---------------------------------------------------------- MMA waiter
        int s = 0, ab = 0, h = 0;
        uint32_t ph = 0, aph = 0;
        bool dead = false;
        for (int t = first; t < n_tiles; t += step) {
            if (lane == 0) {
                if (!dead && *abort_flag) dead = true;
                if (!dead && !tc::mbar_wait_spin(&acce[ab], aph ^ 1u, lim)) { expired(); dead = true; }
                go_flag[h & 1] = dead ? 0 : 1;
            }
            if ((ab ^= 1) == 0) aph ^= 1u;
            __syncwarp();
            tc::named_bar_sync(kHandoffBar, 64);
            const bool go = go_flag[h & 1] != 0;
            ++h;
            if (!go) break;
            for (int kb = 0; kb < p.nkb; ++kb) {
                if (lane == 0) {
                    if (!dead && *abort_flag) dead = true;
                    if (!dead && !tc::mbar_wait_spin(&full[s], ph, lim)) { expired(); dead = true; }
                }
                __syncwarp();
                tc::named_bar_sync(kHandoffBar, 64);
                if (++s == S) { s = 0; ph ^= 1u; }
            }
        }
        __syncwarp();
        __syncthreads();
    } else {
        // ---------------------------------------------------------- epilogue
        // Lane 32 q + i of an accumulator holds weight row m * 128 + 32 q + i.
        // Neighbouring lanes exchange one of every two rows' values, so that a
        // lane stores two features of one row and a warp 64 bytes of two rows:
        // no shared memory, whose latency the MMAs raise.
        const int q = warp & 3, part = (warp - kEpiWarp) >> 2;
        bool dead = false;
        int ab = 0;
        uint32_t fph = 0;
        for (int t = first; t < n_tiles; t += step) {
            const int nrows = w.nrows, odd = lane & 1;
            const int f = w.m * 128 + 32 * q + (lane & ~1);
            __nv_bfloat16* out = p.y + (long long)(w.row0 + odd) * p.ldy + f;
            w.next(gr, p.E, p.m_total);
            if (warp == kEpiWarp && lane == 0) {   // one poller; an expiry leaves undefined outputs and a status
                if (!dead && *abort_flag) dead = true;
                if (!dead && !tc::mbar_wait_spin(&accf[ab], fph, lim)) { expired(); dead = true; }
            }
            __syncwarp();
            tc::named_bar_sync(kEpiBar, 32 * Sh::kEpiWarps);
            tc::tc_fence_after();
            for (int c0 = 16 * part; c0 < nrows; c0 += 4 * Sh::kEpiWarps) {
                float v[16];
                tc::tmem_ld16(tbase + ab * BN + (static_cast<uint32_t>(32 * q) << 16) + c0, v);
                __nv_bfloat16* o = out + (long long)c0 * p.ldy;
                const int left = f < p.N ? nrows - c0 - odd : 0;
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float got = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[i + 1], 1);
                    const __nv_bfloat162 h = odd ? __floats2bfloat162_rn(got, v[i + 1]) : __floats2bfloat162_rn(v[i], got);
                    if (i < left) *reinterpret_cast<__nv_bfloat162*>(o + (uint32_t)i * (uint32_t)p.ldy) = h;
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&acce[ab]);
            ab ^= 1;
            if (ab == 0) fph ^= 1u;
        }
        __syncthreads();
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tbase, Sh::kCols);
    }
    pdl_wait();   // also a CTA without tiles ends after the kernel before this one
}

constexpr int kMaxDevices = 64;
__device__ int g_expiries;
int* g_expiries_ptr[kMaxDevices] = {};
int g_sms[kMaxDevices] = {};
// Test hooks: of the thread that sets them, for the calls it makes.
thread_local long long t_wait_limit = 0;
thread_local int t_stall = 0;

int current_device() {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kMaxDevices ? dev : -1;
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

template <int BN>
int set_attributes() {
    return qbh::cuda_err(cudaFuncSetAttribute(k_mx_product<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              Shape<BN>::smem(QBMOE_MAX_EXPERTS)));
}

template <int BN>
int launch(const qbh::MxProduct& q, Params& p, cudaStream_t s) {
    for (int i = 0; i < Shape<BN>::kBoxes; ++i)
        if (!qbh::encode_rows(&p.b[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, q.x_codes, q.R, q.K / 2, q.K / 2, 128,
                              Shape<BN>::kBox * (i + 1)))
            return QBMOE_ECUDA;
    if (p.sf_tma && !qbh::encode_rows(&p.b_sf, CU_TENSOR_MAP_DATA_TYPE_UINT8, q.x_scales, q.R, q.K / 32, q.K / 32, 16, BN,
                                      true))
        return QBMOE_ECUDA;
    // row tiles of all experts: at most one ragged tile for each that has rows
    const long long tiles = ((long long)(q.R / BN) + min(q.E, q.R)) * p.m_total;
    const int grid = (int)min(tiles, (long long)qbh::sm_count() * (BN == 16 ? 2 : 1));
    const size_t smem = Shape<BN>::smem(q.E);
    if (q.raw) {
        // the product may set itself up, and load weights, while its rows are quantised
        const int rc = qbh::mx_quantize(q.R, q.K, q.raw_type, q.raw, q.raw_ld, q.x_codes, q.x_scales, nullptr, s);
        if (rc) return rc;
        return qbh::launch_pdl(k_mx_product<BN>, dim3(grid), dim3(Shape<BN>::kThreads), smem, s, p);
    }
    k_mx_product<BN><<<grid, Shape<BN>::kThreads, smem, s>>>(p);
    return qbh::cuda_err(cudaGetLastError());
}

}  // namespace

namespace qbh {

int mx_product_init() {
    const int dev = current_device();
    if (dev < 0) return QBMOE_ECUDA;
    void* f = nullptr;
    int rc = cuda_err(cudaGetSymbolAddress(&f, g_expiries));
    if (!rc) rc = cuda_err(cudaDeviceGetAttribute(&g_sms[dev], cudaDevAttrMultiProcessorCount, dev));
    if (!rc) rc = set_attributes<16>();
    if (!rc) rc = set_attributes<64>();
    if (!rc) rc = set_attributes<128>();
    if (!rc) rc = set_attributes<192>();
    if (!rc) rc = set_attributes<208>();
    if (!rc) g_expiries_ptr[dev] = static_cast<int*>(f);
    return rc;
}

int* mx_expiries() {
    const int dev = current_device();
    return dev < 0 ? nullptr : g_expiries_ptr[dev];
}
int mx_new_expiries(cudaStream_t s) {
    int* p = mx_expiries();
    if (!p) return QBMOE_OK;   // no call has run on this device
    // how often a wait had expired when this thread last asked; the count is never
    // reset, so that no thread takes another's answer
    thread_local int t_seen[kMaxDevices] = {};
    int v = 0;
    if (cudaMemcpyAsync(&v, p, 4, cudaMemcpyDeviceToHost, s) != cudaSuccess) return QBMOE_ECUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return QBMOE_ECUDA;
    int& seen = t_seen[current_device()];
    const int rc = v == seen ? QBMOE_OK : QBMOE_ETIMEOUT;
    seen = v;
    return rc;
}
long long mx_wait_limit() { return t_wait_limit; }
void mx_set_wait_limit(long long polls) { t_wait_limit = polls > 0 ? polls : 0; }
int mx_stall() { return t_stall; }
void mx_set_stall(int on) { t_stall = on; }
int sm_count() {
    const int dev = current_device();
    return dev < 0 || g_sms[dev] < 1 ? 1 : g_sms[dev];
}

bool encode_rows(CUtensorMap* m, CUtensorMapDataType type, const void* base, long long rows, long long cols,
                 long long ld_bytes, int box_cols, int box_rows, bool plain) {
    const auto encode = encoder();
    if (!encode) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld_bytes};
    cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    cuuint32_t es[2] = {1, 1};
    return encode(m, type, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  plain                                                                  ? CU_TENSOR_MAP_SWIZZLE_NONE
                  : type == CU_TENSOR_MAP_DATA_TYPE_UINT8 && box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                                            : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int mx_product(const MxProduct& q, cudaStream_t s) {
    Params p{};
    if (!encode_rows(&p.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, q.w_codes, (long long)q.E * q.N, q.K / 2, q.K / 2, 128, 128))
        return QBMOE_ECUDA;
    p.sf_tma = q.K % 512 == 0;
    if (p.sf_tma && !encode_rows(&p.a_sf, CU_TENSOR_MAP_DATA_TYPE_UINT8, q.w_scales, (long long)q.E * q.N, q.K / 32,
                                 q.K / 32, 16, 128, true))
        return QBMOE_ECUDA;
    p.a_sc = q.w_scales;
    p.b_sc = q.x_scales;
    p.offsets = q.offsets;
    p.y = static_cast<__nv_bfloat16*>(q.y);
    p.ldy = q.ldy;
    p.R = q.R; p.E = q.E; p.N = q.N; p.K = q.K;
    p.nkb = (q.K + kStageK - 1) / kStageK;
    p.m_total = (q.N + 127) / 128;
    p.sf_bytes = q.K % 256 == 0 ? 8 : q.K % 128 == 0 ? 4 : 1;
    p.weights_ready = q.raw != nullptr;
    p.expiries = mx_expiries();
    p.wait_limit = t_wait_limit;
    p.stall = t_stall;
    // Row tile: the smallest that holds an average expert's rows, 192 beyond. One
    // matrix whose tiles of 208 rows save over a quarter of the grid's rounds takes those (by
    // 3584 x 7168, 1040 rows, one round or two: 23.2 against 27.3 us; 1999 rows, two
    // or three: 31.4 against 33.5).
    const auto rounds = [&](int rows) {
        const long long tiles = (long long)((q.R + rows - 1) / rows) * p.m_total;
        return (tiles + sm_count() - 1) / sm_count();
    };
    const int avg = (q.R + q.E - 1) / q.E;
    if (avg <= 16) return launch<16>(q, p, s);
    if (avg <= 64) return launch<64>(q, p, s);
    if (avg <= 128) return launch<128>(q, p, s);
    if (q.E > 1 || 4 * rounds(208) >= 3 * rounds(192)) return launch<192>(q, p, s);
    return launch<208>(q, p, s);
}

}  // namespace qbh
