// Gradients of the MXFP4 product on the tensor cores of sm_103a.
//
//   rows     dx[r][k]    = sum_f dy[r][f] w[e][f][k]     (contraction over f)
//   weights  dw[e][f][k] = sum_(r of e) dy[r][f] x[r][k] (contraction over the expert's rows)
//
// Both are D[k][j] = sum_c Q[c][k] dy(c, j) with an MXFP4 matrix Q [contraction,
// K] and the bf16 gradient: an E2M1 code times a power of two is a bf16 number,
// so decoding Q is exact and the products (kind::f16, fp32 accumulation) are
// those of the formulas.  Q is the MMA's A operand (M = 128 columns of K, which
// lie along memory: MN-major) and dy its B operand (N <= 256 rows for dx,
// K-major; features for dw, MN-major): what is decoded once serves 256 columns
// of the other side, and a warp's 32 lanes hold 32 consecutive k of an output row.
// (With Q as the N = 256 side the decoding took 3900 instructions a stage and
// bound the kernel at 1900 cycles a stage.)
//
// One persistent warp-specialised kernel, stages of 64 contraction steps:
//   warp 0       TMA of dy (one lane); it alone waits for a free slot and then
//                meets the slot's converters at a named barrier.  (A suspended
//                mbarrier wait takes about a microsecond to come back, and every
//                warp that polls instead slows the others: dx 692 us with each
//                converter warp polling, 1190 us with each suspended.)
//   warp 1       TMEM owner and MMA issuer (one lane), warp 2 its waiter
//   warps 3+     converters, two or four warps for each slot of the ring: codes and
//                scales, which each warp copies by TMA to a buffer of its own a slot's
//                turn ahead, to bf16 in the swizzled A tile.  Decoding a stage is mostly
//                latency, so the stages in the ring are decoded side by side.  (Loads
//                of the same lead from global memory to registers: dx 496 instead of 424
//                us, dw 728 instead of 680.)
//   the rest     epilogue, one per lane quarter: TMEM -> registers -> 64 or
//                128 bytes of a row per store
// A weight gradient's last stage may reach past its expert's rows, where another
// expert's gradient may be infinite, and 0 * inf is not 0: whole groups of 16 rows
// come by TMA, the converters write the last group with zeros past the end, and
// groups beyond it are not multiplied.
// The tensor cores' fp32 accumulation drops low bits: its error grows with the
// number of steps (6.8e-6 of dw's norm over 40000 rows, where fp32 additions lose
// 1e-7).  An fp32 weight gradient therefore takes its rows kSegRows at a time:
// the epilogue adds each later segment to what it stored for the ones before.
// Where there are fewer tiles than SMs, an expert's rows are also cut into
// parts for different CTAs, summed in order by a second kernel.
//
// Measured (65536 rows over 224 experts, 1024 x 3584): dx 424 us, 640 cycles a stage
// of which the MMAs are 330: the hand-offs between the warps bound it; dw in fp32
// 680 us, 3.3 GB of stores, which alone take 500.
#include "mxfp4.cuh"
#include "mxfp4_decode.cuh"
#include "tc_ptx.cuh"

namespace {

using namespace qb;

constexpr int kM = 128, kN = 256, kC = 64;           // tile of D, contraction steps per stage
constexpr int kABytes = kM * kC * 2, kBBytes = kN * kC * 2;
static_assert(kN == 256, "the last, partial group of dy rows is written as 32 chunks of 8 features");
constexpr int kBlockBytes = kC * 128;                // 64 columns x 64 steps of an MN-major tile
constexpr int kBox = 64;                             // heights of the row-tile maps: 64, 128, 192, 256
constexpr long long kSms = 152;
constexpr int kSegRows = 4096;                       // rows accumulated on the tensor cores alone (fp32 dw)
constexpr int kStages = 4;
constexpr int kConvWarp = 3;
// Warps by direction.  dx: 16 converters decode a slot in half the latency of 8
// (424 against 441 us).  dw needs more registers a converter (the tail of dy), and spills
// with 16 (760 against 680 us).  8 epilogue warps gain neither (dx 430, dw 750).
template <bool kWeights>
struct Warps {
    static constexpr int kConv = kWeights ? 8 : 16, kEpi = 4;
    static constexpr int kEpiFirst = kConvWarp + kConv;
    static constexpr int kConvPer = kConv / kStages;           // warps of a slot
    static constexpr int kItems = kC * 4 / (32 * kConvPer);    // 32-column blocks a thread decodes
    static constexpr int kThreads = (kEpiFirst + kEpi) * 32;
};
constexpr int kRawBytes = kC * kM / 2, kRawScales = kC * 16;   // codes and scales (16 bytes a row) of a stage
constexpr int kMmaWarp = 1, kWaitWarp = 2;
constexpr int kHandoffBar = 1, kEpiBar = 2, kSlotBar = 3;   // kSlotBar + slot
constexpr long long kDefaultWait = 1LL << 17;
constexpr long long kDrainWait = 1LL << 12;

struct Params {
    CUtensorMap b[4];            // dy [R, N] bf16: boxes of 64 features x 64 i rows; weights: x 64 and x 16 rows
    CUtensorMap q, q_sf;         // Q's codes [., K / 2] and, if sf_tma, scales [., K / 32]: a converter warp's rows
    int sf_tma;
    const __nv_bfloat16* dy;
    long long lddy;
    const uint8_t* scales;
    const int32_t* offsets;
    void* out;
    long long ldo;
    int R, E, N, K;
    int k_tiles, f_tiles, f_per; // 128-column tiles of K; weights: tiles of N and features in each
    int splits;                  // weights: parts of each expert's rows, out [splits, E, N, K]
    int seg_rows;                // weights: rows per accumulation
    int step_e, step_s, step_f, step_k;   // weights: the grid size in experts, parts and tiles
    int* expiries;
    long long wait_limit;
    int stall;
};

constexpr int smem_bytes(int E) {
    return 1024 + kStages * (kABytes + kBBytes + kRawBytes + kRawScales) + (2 * (E + 1) + 64) * 4 + 512;
}

// One tile of D: columns kt * 128 .. of K for the output rows [row0, row0 + cols)
// (rows of dx, features of dw), and its contraction: `len` steps from Q row `q0`.
struct Tile {
    int e, row0, cols, kt, len;
    long long q0;    // (weights: b0)
    int b0;          // weights: first row of dy and of Q
    bool first;      // nothing is stored for this tile yet
};
template <bool kWeights>
struct Tiles {
    Walker<kN> w;      // rows
    int e, part, ft, kt;   // weights: expert, part of its rows, feature tile, column tile (fastest)
    int r0, r1;            // weights: rows of the part that are still to do
    bool first;
    int t;
    QB_DEV int count(const Params& p, const Groups& gr) const {
        return kWeights ? p.E * p.splits * p.f_tiles * p.k_tiles : gr.toff[p.E] * p.k_tiles;
    }
    QB_DEV void range(const Params& p, const Groups& gr) {
        if (e >= p.E) return;   // past the last tile
        const int a = gr.seg[e], len = max(gr.seg[e + 1] - a, 0);
        r0 = a;
        r1 = a + len;
        if (p.splits > 1) {
            const long long per = (len / p.splits + kC) / kC * kC;
            r0 = a + (int)min((long long)len, part * per);
            r1 = a + (int)min((long long)len, (part + 1) * per);
        }
        first = true;
    }
    QB_DEV void start(const Params& p, const Groups& gr) {
        t = blockIdx.x;
        if (kWeights) {
            int rest = t / p.k_tiles;
            kt = t - rest * p.k_tiles;
            ft = rest % p.f_tiles;
            rest /= p.f_tiles;
            part = rest % p.splits;
            e = rest / p.splits;
            range(p, gr);
        } else {
            w.start(gr, p.E, p.k_tiles);
        }
    }
    QB_DEV void next(const Params& p, const Groups& gr) {
        if (kWeights) {
            if (r1 - r0 > p.seg_rows) {   // the same tile's next rows
                r0 += p.seg_rows;
                first = false;
                return;
            }
            t += gridDim.x;   // the grid's stride in (e, part, ft, kt), with carries
            kt += p.step_k;
            ft += p.step_f;
            part += p.step_s;
            e += p.step_e;
            if (kt >= p.k_tiles) kt -= p.k_tiles, ++ft;
            if (ft >= p.f_tiles) ft -= p.f_tiles, ++part;
            if (part >= p.splits) part -= p.splits, ++e;
            range(p, gr);
        } else {
            t += gridDim.x;
            w.next(gr, p.E, p.k_tiles);
        }
    }
    QB_DEV Tile get(const Params& p, const Groups& gr) const {
        Tile x;
        if (kWeights) {
            x.e = part * p.E + e;   // of the output
            x.kt = kt;
            x.row0 = ft * p.f_per;
            x.cols = min(p.f_per, p.N - x.row0);
            x.b0 = r0;
            x.len = min(r1 - r0, p.seg_rows);
            x.first = first;
        } else {
            x.e = w.g;
            x.kt = w.m;
            x.row0 = w.row0;
            x.cols = w.nrows;
            x.len = p.N;
            x.q0 = (long long)w.g * p.N;
            x.b0 = 0;
            x.first = true;
        }
        return x;
    }
};

// A slot's stages: every kStages-th of the CTA's sequence of (tile, stage) pairs.
template <bool kWeights>
struct Cursor {
    Tiles<kWeights> it;
    Tile x;
    int c;        // first contraction step of the stage
    bool live;
    QB_DEV void start(const Params& p, const Groups& gr, int n_tiles, const Tiles<kWeights>& from, int slot) {
        it = from;
        live = it.t < n_tiles;
        if (live) x = it.get(p, gr);
        c = 0;
        advance(p, gr, n_tiles, slot);
    }
    QB_DEV void advance(const Params& p, const Groups& gr, int n_tiles, int stages) {
        c += stages * kC;
        while (live && c >= x.len) {
            c -= (x.len + kC - 1) / kC * kC;
            it.next(p, gr);
            live = it.t < n_tiles;
            if (live) x = it.get(p, gr);
        }
    }
};

// MN-major tile, 128-byte swizzle: 64-column blocks of [64 steps][128 bytes].
// Leading offset: from one block of 64 columns to the next; stride offset:
// from 8 contraction steps to the next 8.
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(kBlockBytes >> 4) << 16) |
           (static_cast<uint64_t>(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// 16-byte chunk (8 columns) `chunk` of contraction step c, in bytes.
__device__ __forceinline__ int mn_offset(int c, int chunk) {
    return (chunk >> 3) * kBlockBytes + c * 128 + (((chunk & 7) ^ (c & 7)) << 4);
}

// (32-bit shared addresses: the converters are short of registers.)
__device__ __forceinline__ void st_shared16(uint32_t addr, const uint4& v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_shared_byte(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
// (Straight into a 32-bit register: a conversion would wait for the load.)
__device__ __forceinline__ uint32_t ld_byte(const uint8_t* p) {
    uint32_t v;
    asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

template <bool kWeights, typename Out>
__global__ void __launch_bounds__(Warps<kWeights>::kThreads, 1) k_mx_grad(const __grid_constant__ Params p) {
    constexpr int kConvPer = Warps<kWeights>::kConvPer, kItems = Warps<kWeights>::kItems;
    constexpr int kEpiWarp = Warps<kWeights>::kEpiFirst, kEpiWarps = Warps<kWeights>::kEpi;
    constexpr int kThreads = Warps<kWeights>::kThreads;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* a_ring = smem;
    uint8_t* b_ring = a_ring + kStages * kABytes;
    uint8_t* raw_codes = b_ring + kStages * kBBytes;           // a part for each converter warp
    uint8_t* raw_scales = raw_codes + kStages * kRawBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(raw_scales + kStages * kRawScales);
    uint64_t* empty = full + kStages;
    uint64_t* accf = empty + kStages;
    uint64_t* acce = accf + 2;
    uint64_t* drain = acce + 2;
    uint64_t* raw = drain + 1;                                 // [converter warps]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(raw + Warps<kWeights>::kConv + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* go_flag = reinterpret_cast<volatile int*>(tmem_slot + 2);   // [2]
    int* scratch = reinterpret_cast<int*>(tmem_slot + 4);                     // [kThreads / 32]
    Groups gr;
    gr.seg = scratch + 32;
    gr.toff = gr.seg + p.E + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long lim = p.wait_limit > 0 ? p.wait_limit : kDefaultWait;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(&full[s], 1 + kConvPer);
            tc::mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            tc::mbar_init(&accf[a], 1);
            tc::mbar_init(&acce[a], kEpiWarps);
        }
        tc::mbar_init(drain, 1);
        for (int i = 0; i < Warps<kWeights>::kConv; ++i) tc::mbar_init(&raw[i], 1);
        *abort_flag = 0;
        tc::fence_mbar_init();
        tc::fence_proxy_async_smem();
        tc::prefetch_tmap(&p.b[0]);
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(tmem_slot, 512);   // two accumulators of 256 columns
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    load_groups<kN, kThreads>(gr, p.offsets, p.E, p.R, scratch);
    tc::tc_fence_after();
    const uint32_t tbase = *tmem_slot;
    Tiles<kWeights> it;
    const int n_tiles = it.count(p, gr);
    it.start(p, gr);
    auto expired = [&] {
        if (p.expiries) atomicAdd(p.expiries, 1);
        *abort_flag = 1;
    };

    if (warp == 0) {
        // ---------------------------------------------------------- TMA of dy
        uint32_t issued = 0, last_par = 0;
        int s = 0;
        uint32_t ph = 0;
        bool dead = false;   // lane 0: an expiry; only the meetings go on
        for (; it.t < n_tiles; it.next(p, gr)) {
            const Tile x = it.get(p, gr);
            const int box = (x.cols - 1) / kBox, blocks = (x.cols + 63) / 64;
            if (lane == 0 && *abort_flag) dead = true;
            for (int c0 = 0; c0 < x.len; c0 += kC) {
                if (lane == 0 && !dead && !tc::mbar_wait_spin(&empty[s], ph ^ 1u, lim)) { expired(); dead = true; }
                if (lane == 0 && !dead) {
                    uint8_t* B = b_ring + s * kBBytes;
                    if (!kWeights) {
                        tc::mbar_expect_tx(&full[s], (box + 1) * kBox * 128);
                        tc::tma_load_2d(B, &p.b[box], &full[s], c0, x.row0);
                    } else if (x.len - c0 >= kC) {
                        tc::mbar_expect_tx(&full[s], blocks * kBlockBytes);
                        for (int i = 0; i < blocks; ++i)
                            tc::tma_load_2d(B + i * kBlockBytes, &p.b[0], &full[s], x.row0 + 64 * i, x.b0 + c0);
                    } else {   // whole groups of 16 rows; the converters write the rest
                        const int groups = (x.len - c0) / 16;
                        tc::mbar_expect_tx(&full[s], blocks * groups * 2048);
                        for (int i = 0; i < blocks; ++i)
                            for (int h = 0; h < groups; ++h)
                                tc::tma_load_2d(B + i * kBlockBytes + h * 2048, &p.b[1], &full[s], x.row0 + 64 * i,
                                                x.b0 + c0 + 16 * h);
                    }
                    issued |= 1u << s;
                    last_par = (last_par & ~(1u << s)) | (ph << s);
                }
                __syncwarp();
                tc::named_bar_sync(kSlotBar + s, 32 + 32 * kConvPer);
                if (++s == kStages) { s = 0; ph ^= 1u; }
            }
        }
        __syncthreads();
        if (lane == 0 && *abort_flag)
            for (int i = 0; i < kStages; ++i)
                if ((issued >> i) & 1u) tc::mbar_wait(&full[i], (last_par >> i) & 1u, kDrainWait);
    } else if (warp >= kConvWarp && warp < kEpiWarp) {
        // ---------------------------------------------------------- converters
        // A warp has 8 kItems consecutive steps of its slot's stages, a thread (c, b) of
        // them steps c, c + 8, .. and column block b (32 columns, one scale); eight
        // consecutive lanes have eight rows, whose 16-byte chunks the swizzles put in
        // eight different places.  Once a stage's codes are in registers the copy of
        // the next turn's may overwrite them.  Scales come with them where their rows
        // are 16-byte multiples, by plain loads otherwise.
        const int slot = (warp - kConvWarp) / kConvPer, team = (warp - kConvWarp) % kConvPer;
        const int ct = threadIdx.x - (kConvWarp + slot * kConvPer) * 32;
        constexpr int kRows = 8 * kItems;
        static_assert(kRows * kConvPer == kC);
        const int b = lane >> 3, c = team * kRows + (lane & 7);
        uint64_t* arrived = &raw[warp - kConvWarp];
        uint8_t* my_codes = raw_codes + (warp - kConvWarp) * (kRows * 64);
        uint8_t* my_scales = raw_scales + (warp - kConvWarp) * (kRows * 16);
        // row i of 64 bytes: chunk b is at b ^ (i / 2 % 4)
        const uint32_t code_at = tc::smem_u32(my_codes) + (lane & 7) * 64 + ((b ^ ((lane & 7) >> 1)) << 4);
        const uint32_t scale_at = tc::smem_u32(my_scales) + (lane & 7) * 16 + b;
        const int pitch = p.K / 32;
        Cursor<kWeights> cur;
        cur.start(p, gr, n_tiles, it, slot);
        uint32_t sc[kItems];
        // the last, partial group of 16 rows of dy: 16 steps x 32 chunks of 8 features
        constexpr int kTail = 16 * 32 / (32 * kConvPer);
        uint4 bv[kWeights ? kTail : 1];
        int rem = 0;     // its rows
        int left = 0;    // steps from this thread's first to the end of the tile
        bool dead = false, asked = false;   // lane 0: an expiry; a copy is on its way
        uint32_t ph = 0;
        auto first_row = [&] { return (int)((kWeights ? (long long)cur.x.b0 : cur.x.q0) + cur.c + team * kRows); };
        auto ask = [&] {
            if (cur.live && lane == 0 && !dead) {
                const int k = cur.x.kt * kM, row = first_row();
                tc::mbar_expect_tx(arrived, kRows * (p.sf_tma ? 80 : 64));
                tc::tma_load_2d(my_codes, &p.q, arrived, k / 2, row);
                if (p.sf_tma) tc::tma_load_2d(my_scales, &p.q_sf, arrived, k / 32 & ~15, row);
                asked = true;
            }
        };
        auto fetch = [&] {   // the rest of a stage
            if (!cur.live) return;
            left = cur.x.len - cur.c - c;
            if (!p.sf_tma) {
                const int k = cur.x.kt * kM;
                const uint8_t* scales = p.scales + ((long long)first_row() + (lane & 7)) * pitch + k / 32 + b;
#pragma unroll
                for (int i = 0; i < kItems; ++i) {
                    sc[i] = 127;
                    if (8 * i < left && k + 32 * b < p.K) sc[i] = ld_byte(scales + i * (8 * pitch));
                }
            }
            if constexpr (kWeights) {
                rem = cur.x.len - cur.c < kC ? cur.x.len & 15 : 0;
                if (rem) {
                    const int f = cur.x.row0 + 8 * (ct & 31);
#pragma unroll
                    for (int i = 0; i < kTail; ++i) {
                        const int h = (ct >> 5) + kConvPer * i;
                        bv[i] = h < rem && f < p.N
                                    ? __ldg(reinterpret_cast<const uint4*>(
                                          p.dy + (long long)(cur.x.b0 + cur.x.len - rem + h) * p.lddy + f))
                                    : make_uint4(0, 0, 0, 0);
                    }
                }
            }
        };
        ask();
        fetch();
        const uint32_t B = tc::smem_u32(b_ring + slot * kBBytes);
        uint32_t dst[4];   // of the thread's first step; the swizzle repeats every 8 steps
#pragma unroll
        for (int j = 0; j < 4; ++j) dst[j] = tc::smem_u32(a_ring + slot * kABytes + mn_offset(c, 4 * b + j));
        while (cur.live) {
            if (lane == 0 && !dead) {
                if (tc::mbar_wait_spin(arrived, ph, lim)) {
                    asked = false;
                } else {
                    expired();
                    dead = true;
                }
                ph ^= 1u;
            }
            __syncwarp();
            uint4 v[kItems];
            const uint32_t first_scale = scale_at + ((cur.x.kt & 3) << 2);
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                v[i] = ld_shared16(code_at + i * 512);
                if (p.sf_tma) sc[i] = ld_shared_byte(first_scale + i * 128);
                if (8 * i >= left) v[i] = make_uint4(0, 0, 0, 0), sc[i] = 127;   // another expert's rows
            }
            tc::named_bar_sync(kSlotBar + slot, 32 + 32 * kConvPer);   // the slot is free, the codes are read
            if constexpr (kWeights) {
                if (rem) {
                    const int h0 = (cur.x.len - cur.c) & ~15;
#pragma unroll
                    for (int i = 0; i < kTail; ++i)
                        st_shared16(B + mn_offset(h0 + (ct >> 5) + kConvPer * i, ct & 31), bv[i]);
                }
            }
            cur.advance(p, gr, n_tiles, kStages);
            ask();
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                const uint32_t q[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                const __nv_bfloat162 factor = mx_factor(sc[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t o[4];
                    mx_decode_pairs(q[j], factor, o);
                    if (sc[i] >= kMxLargeScale) mx_rescale(sc[i], o);
                    st_shared16(dst[j] + i * 1024, make_uint4(o[0], o[1], o[2], o[3]));
                }
            }
            tc::fence_proxy_async_smem();   // generic-proxy writes -> tcgen05.mma reads
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&full[slot]);
            fetch();
        }
        if (lane == 0 && asked) tc::mbar_wait(arrived, ph ^ 1u, kDrainWait);
        __syncthreads();
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------- MMA issuer
        int s = 0, ab = 0, h = 0;
        // A (and for dw B) MN-major: bit 15 (16); 16 steps are two 8-step groups of
        // 1024 bytes when MN-major, 32 bytes of a row when K-major
        const uint32_t major = (1u << 15) | (kWeights ? 1u << 16 : 0u);
        const uint64_t a0 = desc_mn(tc::smem_u32(a_ring));
        const uint64_t b0 = kWeights ? desc_mn(tc::smem_u32(b_ring)) : tc::desc_sw128(tc::smem_u32(b_ring));
        constexpr uint64_t kAStep = 2048 >> 4, kBStep = kWeights ? 2048 >> 4 : 32 >> 4;
        const int first = it.t;
        for (; it.t < n_tiles; it.next(p, gr)) {
            const Tile x = it.get(p, gr);
            tc::named_bar_sync(kHandoffBar, 64);
            const bool go = go_flag[h & 1] != 0;
            ++h;
            if (!go) break;
            const uint32_t d = tbase + ab * kN;
            const uint32_t idesc = tc::idesc_bf16_m128((x.cols + 15) & ~15) | major;
            for (int c0 = 0; c0 < x.len; c0 += kC) {
                tc::named_bar_sync(kHandoffBar, 64);
                if (tc::elect_one()) {
                    tc::tc_fence_after();
                    const uint64_t ad = a0 + (uint64_t)(s * (kABytes >> 4)), bd = b0 + (uint64_t)(s * (kBBytes >> 4));
                    const int left = x.len - c0;
                    tc::tc_mma_bf16(d, ad, bd, idesc, c0 != 0);
                    if (left > 16) tc::tc_mma_bf16(d, ad + kAStep, bd + kBStep, idesc, 1);
                    if (left > 32) tc::tc_mma_bf16(d, ad + 2 * kAStep, bd + 2 * kBStep, idesc, 1);
                    if (left > 48) tc::tc_mma_bf16(d, ad + 3 * kAStep, bd + 3 * kBStep, idesc, 1);
                    tc::tc_commit(&empty[s]);
                }
                __syncwarp();
                if (++s == kStages) s = 0;
            }
            if (tc::elect_one() && !(p.stall && it.t == first)) tc::tc_commit(&accf[ab]);
            __syncwarp();
            ab ^= 1;
        }
        if (tc::elect_one()) {
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
        for (; it.t < n_tiles; it.next(p, gr)) {
            const Tile x = it.get(p, gr);
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
            for (int c0 = 0; c0 < x.len; c0 += kC) {
                if (lane == 0) {
                    if (!dead && *abort_flag) dead = true;
                    if (!dead && !tc::mbar_wait_spin(&full[s], ph, lim)) { expired(); dead = true; }
                }
                __syncwarp();
                tc::named_bar_sync(kHandoffBar, 64);
                if (++s == kStages) { s = 0; ph ^= 1u; }
            }
        }
        __syncwarp();
        __syncthreads();
    } else {
        // ---------------------------------------------------------- epilogue
        // Lane 32 q + i of an accumulator is a column of kt * 128 + 32 q .. + 31 of K, in
        // the order in which the converters decode a word: lanes 2 j and 2 j + 1 of
        // eight are columns j and j + 4.  Its TMEM columns are output rows.  fp32: a
        // warp stores 128 bytes of a row at a time; bf16: lanes of neighbouring columns
        // exchange one of every two rows' values and a warp stores 64 bytes of two rows.
        const int column = (lane & ~7) | ((lane & 7) >> 1) | ((lane & 1) << 2);
        const int q = warp & 3, odd = (lane >> 1) & 1;
        const uint32_t ldo = (uint32_t)p.ldo;
        bool dead = false;
        int ab = 0;
        uint32_t fph = 0;
        for (; it.t < n_tiles; it.next(p, gr)) {
            const Tile x = it.get(p, gr);
            if (warp == kEpiWarp && lane == 0) {   // one poller; an expiry leaves undefined outputs and a status
                if (!dead && *abort_flag) dead = true;
                if (!dead && !tc::mbar_wait_spin(&accf[ab], fph, lim)) { expired(); dead = true; }
            }
            __syncwarp();
            tc::named_bar_sync(kEpiBar, 32 * kEpiWarps);
            tc::tc_fence_after();
            const long long first_row = kWeights ? (long long)x.e * p.N + x.row0 : x.row0;
            const int k = x.kt * kM + 32 * q;   // K is a multiple of 32: a warp's columns are all there or none
            const int cols = k < p.K ? x.cols : 0;
            Out* out = static_cast<Out*>(p.out) + first_row * p.ldo + k;
            for (int c0 = 0; c0 < cols; c0 += 16) {
                float v[16];
                tc::tmem_ld16(tbase + ab * kN + (static_cast<uint32_t>(32 * q) << 16) + c0, v);
                if (x.len == 0)
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = 0.0f;   // no rows: nothing was accumulated
                Out* o = out + (long long)c0 * p.ldo;
                const int left = cols - c0;
                if constexpr (sizeof(Out) == 4) {
                    o += column;
                    if (!x.first) {     // this thread stored the sum so far
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (i < left) v[i] += o[(uint32_t)i * ldo];
                    }
                    if (left >= 16) {   // no test a row
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[(uint32_t)i * ldo] = v[i];
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (i < left) o[(uint32_t)i * ldo] = v[i];
                    }
                } else {
                    o += column & ~1;
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float got = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[i + 1], 2);
                        const __nv_bfloat162 h =
                            odd ? __floats2bfloat162_rn(got, v[i + 1]) : __floats2bfloat162_rn(v[i], got);
                        if (i + odd < left) *reinterpret_cast<__nv_bfloat162*>(o + (uint32_t)(i + odd) * ldo) = h;
                    }
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
        tc::tmem_dealloc(tbase, 512);
    }
}

template <bool kWeights, typename Out>
int launch(Params& p, long long tiles, cudaStream_t s) {
    const int grid = (int)min(tiles, (long long)qbh::sm_count());
    int rest = grid / p.k_tiles;
    p.step_k = grid % p.k_tiles;
    p.step_f = rest % p.f_tiles;
    rest /= p.f_tiles;
    p.step_s = rest % p.splits;
    p.step_e = rest / p.splits;
    k_mx_grad<kWeights, Out><<<grid, Warps<kWeights>::kThreads, smem_bytes(p.E), s>>>(p);
    return qbh::cuda_err(cudaGetLastError());
}
// out = sum over the parts, in order; four values a thread.
template <typename Out>
__global__ void __launch_bounds__(256) k_sum_parts(const float4* __restrict__ parts, int splits, long long quads,
                                                   Out* __restrict__ out) {
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < quads; i += (long long)gridDim.x * 256) {
        float4 s = __ldg(parts + i);
        for (int j = 1; j < splits; ++j) {
            const float4 v = __ldg(parts + j * quads + i);
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        if constexpr (sizeof(Out) == 4) {
            reinterpret_cast<float4*>(out)[i] = s;
        } else {
            const __nv_bfloat162 h[2] = {__floats2bfloat162_rn(s.x, s.y), __floats2bfloat162_rn(s.z, s.w)};
            reinterpret_cast<uint2*>(out)[i] = *reinterpret_cast<const uint2*>(h);
        }
    }
}

template <bool kWeights, typename Out>
int set_attributes() {
    return qbh::cuda_err(cudaFuncSetAttribute(k_mx_grad<kWeights, Out>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              smem_bytes(QBMOE_MAX_EXPERTS)));
}

}  // namespace

namespace qbh {

int mx_grad_init() {
    int rc = set_attributes<false, __nv_bfloat16>();
    if (!rc) rc = set_attributes<true, float>();
    if (!rc) rc = set_attributes<true, __nv_bfloat16>();
    return rc;
}

// Parts of each expert's rows: as many as there are SMs (152, whatever the device
// says: the order of the sums is part of the result) for each tile, with at
// least four stages of rows an expert on average in each.  (40000 rows, 264 x 544: 10
// tiles, 270 us in one part, 31 us in 15.)
int mx_wgrad_splits(int R, int E, int N, int K) {
    const long long tiles = (long long)E * ((N + kN - 1) / kN) * ((K + kM - 1) / kM);
    return (int)max(1LL, min(kSms / tiles, (long long)R / E / (4 * kC)));
}

int mx_grad(const MxGrad& q, cudaStream_t s) {
    Params p{};
    // no rows: the maps are not used, but their extent may not be 0
    const void* dy = q.R ? q.dy : q.out;
    const int maps = q.weights ? 2 : min(4, (q.R + kBox - 1) / kBox);
    for (int i = 0; i < maps; ++i)
        if (!encode_rows(&p.b[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dy, q.R ? q.R : 1, q.N, q.lddy * 2, 64,
                         q.weights ? (i ? 16 : kC) : kBox * (i + 1)))
            return QBMOE_ECUDA;
    const long long q_rows = q.weights ? q.R : (long long)q.E * q.N;
    const int box = q.weights ? 8 * Warps<true>::kItems : 8 * Warps<false>::kItems;
    // a TMA row is a multiple of 16 bytes
    p.sf_tma = q.K % 512 == 0 && aligned16(q.scales);
    if (q_rows &&
        (!encode_rows(&p.q, CU_TENSOR_MAP_DATA_TYPE_UINT8, q.codes, q_rows, q.K / 2, q.K / 2, 64, box) ||
         (p.sf_tma && !encode_rows(&p.q_sf, CU_TENSOR_MAP_DATA_TYPE_UINT8, q.scales, q_rows, q.K / 32, q.K / 32, 16, box, true))))
        return QBMOE_ECUDA;
    p.dy = static_cast<const __nv_bfloat16*>(q.dy);
    p.lddy = q.lddy;
    p.scales = q.scales; p.offsets = q.offsets;
    p.out = q.out; p.ldo = q.ldo;
    p.R = q.R; p.E = q.E; p.N = q.N; p.K = q.K;
    p.k_tiles = (q.K + kM - 1) / kM;
    p.f_tiles = (q.N + kN - 1) / kN;
    p.f_per = ((q.N + p.f_tiles - 1) / p.f_tiles + 15) & ~15;
    p.splits = q.weights ? mx_wgrad_splits(q.R, q.E, q.N, q.K) : 1;
    // bf16 sums need no more than the tensor cores keep
    p.seg_rows = q.out_type == QBMOE_F32 || p.splits > 1 ? kSegRows : 0x7fffffff;
    p.expiries = mx_expiries();
    p.wait_limit = mx_wait_limit();
    p.stall = mx_stall();
    if (!q.weights) {
        const long long tiles = ((long long)(q.R / kN) + min(q.E, q.R)) * p.k_tiles;
        return launch<false, __nv_bfloat16>(p, tiles, s);
    }
    const long long tiles = (long long)q.E * p.splits * p.f_tiles * p.k_tiles;
    if (p.splits > 1) {
        p.out = q.parts;
        const int rc = launch<true, float>(p, tiles, s);
        if (rc) return rc;
        const long long quads = (long long)q.E * q.N * q.K / 4;
        const int grid = (int)min((quads + 255) / 256, 8LL * sm_count());
        const float4* parts = static_cast<const float4*>(q.parts);
        if (q.out_type == QBMOE_F32)
            k_sum_parts<float><<<grid, 256, 0, s>>>(parts, p.splits, quads, static_cast<float*>(q.out));
        else
            k_sum_parts<__nv_bfloat16><<<grid, 256, 0, s>>>(parts, p.splits, quads, static_cast<__nv_bfloat16*>(q.out));
        return cuda_err(cudaGetLastError());
    }
    return q.out_type == QBMOE_F32 ? launch<true, float>(p, tiles, s) : launch<true, __nv_bfloat16>(p, tiles, s);
}

}  // namespace qbh
