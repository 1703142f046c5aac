// Gradients of the MXFP4 product on the tensor cores of sm_103a.
//
//   rows     dx[r][k]    = sum_f dy[r][f] w[e][f][k]     (contraction over f)
//   weights  dw[e][f][k] = sum_(r of e) dy[r][f] x[r][k] (contraction over the expert's rows)
//
// Both are D[m][n] = sum_c A[c][m] Q[c][n] with the bf16 gradient as A and an
// MXFP4 matrix Q [contraction, K] as B: an E2M1 code times a power of two is a
// bf16 number, so decoding Q is exact and the products (kind::f16, fp32
// accumulation) are those of the formulas.  The codes lie along n in memory,
// so B is an MN-major operand; A is K-major for dx and MN-major for dw.
//
// One persistent warp-specialised kernel, 128 x 256 tiles of D, stages of 64
// contraction steps:
//   warp 0       TMA of A (one lane)
//   warp 1       TMEM owner and MMA issuer (one lane), warp 2 its waiter
//   warps 3-10   converters: codes and scales from global memory (three stages
//                ahead, in registers) to bf16 in the swizzled B tile
//   warps 11-14  epilogue: TMEM -> per-warp transpose in shared memory -> stores
// A weight tile's last stage may reach past its expert's rows: the converters
// then write A too, with zeros past the end (another expert's gradient may be
// infinite, and 0 * inf is not 0).
#include "mxfp4.cuh"
#include "mxfp4_decode.cuh"
#include "tc_ptx.cuh"

namespace {

using namespace qb;

constexpr int kM = 128, kN = 256, kC = 64;           // tile of D, contraction steps per stage
constexpr int kABytes = kM * kC * 2, kBBytes = kN * kC * 2;
constexpr int kBlockBytes = kC * 128;                // 64 columns x 64 steps of an MN-major tile
constexpr int kStages = 4;
constexpr int kConvWarp = 3, kConvWarps = 8, kEpiWarp = kConvWarp + kConvWarps;
constexpr int kThreads = (kEpiWarp + 4) * 32;        // 480
constexpr int kMmaWarp = 1, kWaitWarp = 2;
constexpr int kHandoffBar = 1;
constexpr int kAhead = 3;                            // stages of codes in flight per converter
constexpr int kEpiRow = 36;                          // transpose row: 32 columns, 4 words of padding
constexpr long long kDefaultWait = 1LL << 17;
constexpr long long kDrainWait = 1LL << 12;

struct Params {
    CUtensorMap a;               // dy [R, N] bf16
    const __nv_bfloat16* dy;
    long long lddy;
    const uint8_t* codes;        // Q's codes [., K / 2] and scales [., K / 32]
    const uint8_t* scales;
    const int32_t* offsets;
    void* out;
    long long ldo;
    int R, E, N, K;
    int m_tiles, n_tiles;        // weights: 128-row tiles of N; both: 256-column tiles of K
    int* status;
    long long wait_limit;
    int stall;
};

constexpr int smem_bytes(int E) {
    return 1024 + kStages * (kABytes + kBBytes) + 4 * 32 * kEpiRow * 4 + (2 * (E + 1) + 64) * 4 + 256;
}

// One tile of D: group e, output rows [row0, row0 + rows) or weight rows from
// row0, column tile nt, and its contraction: `len` steps from Q row `q0`.
struct Tile {
    int e, row0, rows, nt, len;
    long long q0;
    int a0;          // weights: first row of dy
};
template <bool kWeights>
struct Tiles {
    Walker<kM> w;
    int t;
    QB_DEV int count(const Params& p, const Groups& gr) const {
        return kWeights ? p.E * p.m_tiles * p.n_tiles : gr.toff[p.E] * p.n_tiles;
    }
    QB_DEV void start(const Params& p, const Groups& gr) {
        t = blockIdx.x;
        if (!kWeights) w.start(gr, p.E, p.n_tiles);
    }
    QB_DEV void next(const Params& p, const Groups& gr) {
        t += gridDim.x;
        if (!kWeights) w.next(gr, p.E, p.n_tiles);
    }
    QB_DEV Tile get(const Params& p, const Groups& gr) const {
        Tile x;
        if (kWeights) {
            const int per = p.m_tiles * p.n_tiles;
            x.e = t / per;
            const int rem = t - x.e * per, mt = rem / p.n_tiles;
            x.nt = rem - mt * p.n_tiles;
            x.row0 = mt * kM;
            x.rows = min(kM, p.N - x.row0);
            x.a0 = gr.seg[x.e];
            x.len = max(gr.seg[x.e + 1] - x.a0, 0);
            x.q0 = x.a0;
        } else {
            x.e = w.g;
            x.nt = w.m;
            x.row0 = w.row0;
            x.rows = w.nrows;
            x.len = p.N;
            x.q0 = (long long)w.g * p.N;
            x.a0 = 0;
        }
        return x;
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

// 32 columns of one step: codes and their scale byte; zeros where there is nothing.
struct Item {
    uint4 q;
    uint32_t sc;
};

template <bool kWeights, typename Out>
__global__ void __launch_bounds__(kThreads, 1) k_mx_grad(const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* a_ring = smem;
    uint8_t* b_ring = a_ring + kStages * kABytes;
    float* epi = reinterpret_cast<float*>(b_ring + kStages * kBBytes);    // [4][32][kEpiRow]
    uint64_t* full = reinterpret_cast<uint64_t*>(epi + 4 * 32 * kEpiRow);
    uint64_t* empty = full + kStages;
    uint64_t* accf = empty + kStages;
    uint64_t* acce = accf + 2;
    uint64_t* drain = acce + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* go_flag = reinterpret_cast<volatile int*>(tmem_slot + 2);   // [2]
    int* scratch = reinterpret_cast<int*>(tmem_slot + 4);                     // [kThreads / 32]
    Groups gr;
    gr.seg = scratch + 16;
    gr.toff = gr.seg + p.E + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long lim = p.wait_limit > 0 ? p.wait_limit : kDefaultWait;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(&full[s], 1 + kConvWarps);
            tc::mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            tc::mbar_init(&accf[a], 1);
            tc::mbar_init(&acce[a], 4);
        }
        tc::mbar_init(drain, 1);
        *abort_flag = 0;
        tc::fence_mbar_init();
        tc::fence_proxy_async_smem();
        tc::prefetch_tmap(&p.a);
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(tmem_slot, 512);   // two accumulators of 256 columns
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    load_groups<kM, kThreads>(gr, p.offsets, p.E, p.R, scratch);
    tc::tc_fence_after();
    const uint32_t tbase = *tmem_slot;
    Tiles<kWeights> it;
    const int n_tiles = it.count(p, gr);
    it.start(p, gr);
    auto expired = [&] {
        set_status(p.status, QBMOE_ETIMEOUT);
        *abort_flag = 1;
    };

    if (warp == 0) {
        // ---------------------------------------------------------- TMA of A
        uint32_t issued = 0, last_par = 0;
        int s = 0;
        uint32_t ph = 0;
        for (; it.t < n_tiles; it.next(p, gr)) {
            const Tile x = it.get(p, gr);
            int stop = 0;
            if (lane == 0) {
                stop = *abort_flag;
                for (int c0 = 0; c0 < x.len && !stop; c0 += kC) {
                    if (!tc::mbar_wait_spin(&empty[s], ph ^ 1u, lim)) { expired(); stop = 1; break; }
                    uint8_t* A = a_ring + s * kABytes;
                    if (kWeights && x.len - c0 < kC) {
                        tc::mbar_arrive(&full[s]);   // the converters write this stage's A
                    } else {
                        tc::mbar_expect_tx(&full[s], kABytes);
                        if (kWeights) {
                            tc::tma_load_2d(A, &p.a, &full[s], x.row0, x.a0 + c0);
                            tc::tma_load_2d(A + kBlockBytes, &p.a, &full[s], x.row0 + 64, x.a0 + c0);
                        } else {
                            tc::tma_load_2d(A, &p.a, &full[s], c0, x.row0);
                        }
                    }
                    issued |= 1u << s;
                    last_par = (last_par & ~(1u << s)) | (ph << s);
                    if (++s == kStages) { s = 0; ph ^= 1u; }
                }
            }
            if (__shfl_sync(0xffffffffu, stop, 0)) break;
        }
        __syncthreads();
        if (lane == 0 && *abort_flag)
            for (int i = 0; i < kStages; ++i)
                if ((issued >> i) & 1u) tc::mbar_wait(&full[i], (last_par >> i) & 1u, kDrainWait);
    } else if (warp >= kConvWarp && warp < kEpiWarp) {
        // ---------------------------------------------------------- converters
        // Thread (r, b) of a stage: steps r and r + 32, column block b (32
        // columns, one scale).  Eight consecutive lanes read 128 bytes of one
        // row; they write their four 16-byte chunks in an order that puts
        // eight different chunk places in each store.
        const int ct = threadIdx.x - kConvWarp * 32;
        const int b = ct & 7, r = ct >> 3;
        const int half = p.K / 2, pitch = p.K / 32;
        Tile x = {};
        Tile fx = {};                 // tile of the next fetch
        Tiles<kWeights> ft = it;
        int fc = 0;                   // its next stage's first step
        bool fetching = ft.t < n_tiles;
        auto settle = [&] {           // to the next stage that exists
            while (fetching && fc >= fx.len) {
                ft.next(p, gr);
                fetching = ft.t < n_tiles;
                fc = 0;
                if (fetching) fx = ft.get(p, gr);
            }
        };
        if (fetching) { fx = ft.get(p, gr); settle(); }
        auto fetch = [&](Item (&v)[2]) {
            const int k = fx.nt * kN + 32 * b;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = fc + r + 32 * i;
                v[i].q = make_uint4(0, 0, 0, 0);
                v[i].sc = 127;
                if (fetching && c < fx.len && k < p.K) {
                    const long long row = fx.q0 + c;
                    v[i].q = __ldg(reinterpret_cast<const uint4*>(p.codes + row * half + k / 2));
                    v[i].sc = __ldg(p.scales + row * pitch + k / 32);
                }
            }
            if (fetching) { fc += kC; settle(); }
        };
        Item buf[kAhead][2];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch(buf[i]);
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (; it.t < n_tiles && ok; it.next(p, gr)) {
            x = it.get(p, gr);
            for (int c0 = 0; c0 < x.len; c0 += kC) {
                const bool own_a = kWeights && x.len - c0 < kC;
                uint4 av[4];
                if (own_a) {   // 64 steps x 16 chunks of 8 columns, four to a thread
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c = (ct >> 4) + 16 * i, f = x.row0 + 8 * (ct & 15);
                        av[i] = c0 + c < x.len && f < p.N
                                    ? __ldg(reinterpret_cast<const uint4*>(p.dy + (x.a0 + c0 + c) * p.lddy + f))
                                    : make_uint4(0, 0, 0, 0);
                    }
                }
                int w = 1;
                if (lane == 0) {
                    w = !*abort_flag && tc::mbar_wait_spin(&empty[s], ph ^ 1u, lim);
                    if (!w && !*abort_flag) expired();
                }
                if (!__shfl_sync(0xffffffffu, w, 0)) { ok = false; break; }
                if (own_a) {
                    uint8_t* A = a_ring + s * kABytes;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<uint4*>(A + mn_offset((ct >> 4) + 16 * i, ct & 15)) = av[i];
                }
                uint8_t* B = b_ring + s * kBBytes;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t q[4] = {buf[0][i].q.x, buf[0][i].q.y, buf[0][i].q.z, buf[0][i].q.w};
                    // word j of the block goes out in turn j ^ (b >> 1)
                    const int sw = b >> 1;
                    if (sw & 1) { uint32_t t = q[0]; q[0] = q[1]; q[1] = t; t = q[2]; q[2] = q[3]; q[3] = t; }
                    if (sw & 2) { uint32_t t = q[0]; q[0] = q[2]; q[2] = t; t = q[1]; q[1] = q[3]; q[3] = t; }
                    const uint32_t sc = buf[0][i].sc;
                    const int c = r + 32 * i;
                    if (sc >= 2 && sc <= 252) {
                        uint32_t th[2], tl[2];
                        mx_tables((int)sc - 127, th, tl);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t o[4];
                            mx_decode_word(q[j], th, tl, o);
                            *reinterpret_cast<uint4*>(B + mn_offset(c, 4 * b + (j ^ sw))) =
                                make_uint4(o[0], o[1], o[2], o[3]);
                        }
                    } else {
                        const float m = e8m0_value(sc);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t o[4];
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                const __nv_bfloat162 v = __floats2bfloat162_rn(e2m1_value(q[j] >> (8 * h)) * m,
                                                                               e2m1_value(q[j] >> (8 * h + 4)) * m);
                                o[h] = *reinterpret_cast<const uint32_t*>(&v);
                            }
                            *reinterpret_cast<uint4*>(B + mn_offset(c, 4 * b + (j ^ sw))) =
                                make_uint4(o[0], o[1], o[2], o[3]);
                        }
                    }
                }
                tc::fence_proxy_async_smem();   // generic-proxy writes -> tcgen05.mma reads
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&full[s]);
                if (++s == kStages) { s = 0; ph ^= 1u; }
#pragma unroll
                for (int i = 0; i + 1 < kAhead; ++i) { buf[i][0] = buf[i + 1][0]; buf[i][1] = buf[i + 1][1]; }
                fetch(buf[kAhead - 1]);
            }
        }
        __syncthreads();
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------- MMA issuer
        int s = 0, ab = 0, h = 0;
        // bf16 x bf16 -> fp32, M = 128, N = 256; bit 15 / 16: A / B MN-major
        const uint32_t idesc = tc::idesc_bf16_m128(kN) | (kWeights ? 1u << 15 : 0u) | (1u << 16);
        const uint64_t a0 = kWeights ? desc_mn(tc::smem_u32(a_ring)) : tc::desc_sw128(tc::smem_u32(a_ring));
        const uint64_t b0 = desc_mn(tc::smem_u32(b_ring));
        // 16 steps: two 8-step groups of 1024 bytes when MN-major, 32 bytes of a row when K-major
        constexpr uint64_t kAStep = kWeights ? 2048 >> 4 : 32 >> 4, kBStep = 2048 >> 4;
        const int first = it.t;
        for (; it.t < n_tiles; it.next(p, gr)) {
            const Tile x = it.get(p, gr);
            tc::named_bar_sync(kHandoffBar, 64);
            const bool go = go_flag[h & 1] != 0;
            ++h;
            if (!go) break;
            const uint32_t d = tbase + ab * kN;
            for (int c0 = 0; c0 < x.len; c0 += kC) {
                tc::named_bar_sync(kHandoffBar, 64);
                if (lane == 0) {
                    tc::tc_fence_after();
                    const uint64_t ad = a0 + (uint64_t)(s * (kABytes >> 4)), bd = b0 + (uint64_t)(s * (kBBytes >> 4));
#pragma unroll
                    for (int kk = 0; kk < kC / 16; ++kk)
                        tc::tc_mma_bf16(d, ad + kAStep * kk, bd + kBStep * kk, idesc, (c0 | kk) != 0);
                    tc::tc_commit(&empty[s]);
                }
                __syncwarp();
                if (++s == kStages) s = 0;
            }
            if (lane == 0 && !(p.stall && it.t == first)) tc::tc_commit(&accf[ab]);
            __syncwarp();
            ab ^= 1;
        }
        if (lane == 0) {
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
        // Lane 32 q + i of an accumulator is output row 32 q + i.  A warp turns
        // 32 rows x 32 columns around in its piece of shared memory and stores
        // whole row segments.
        const int q = warp & 3;
        float* st = epi + q * 32 * kEpiRow;
        constexpr int kPer = 16 / sizeof(Out);             // columns of a 16-byte store
        constexpr int kLanes = 32 / kPer;                  // lanes of a row segment
        const int sub = lane / kLanes, col = (lane % kLanes) * kPer;
        int ab = 0;
        uint32_t fph = 0;
        for (; it.t < n_tiles; it.next(p, gr)) {
            const Tile x = it.get(p, gr);
            int ok = 1;
            if (lane == 0) {
                ok = tc::mbar_wait(&accf[ab], fph, lim);
                if (!ok) expired();
            }
            if (!__shfl_sync(0xffffffffu, ok, 0)) break;
            tc::tc_fence_after();
            const long long first_row = kWeights ? (long long)x.e * p.N + x.row0 : x.row0;
            const int cols = min(kN, p.K - x.nt * kN);
            Out* out = static_cast<Out*>(p.out) + (first_row + 32 * q) * p.ldo + (long long)x.nt * kN;
            const int rows = x.rows - 32 * q;              // of this warp's 32
            for (int c0 = 0; c0 < cols && rows > 0; c0 += 32) {   // K is a multiple of 32
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    float v[16];
                    tc::tmem_ld16(tbase + ab * kN + (static_cast<uint32_t>(32 * q) << 16) + c0 + 16 * g, v);
                    if (x.len == 0)
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = 0.0f;   // no rows: nothing was accumulated
                    if (g == 0) __syncwarp();                       // the last chunk's readers are done
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<float4*>(st + lane * kEpiRow + 16 * g + 4 * i) =
                            make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                }
                __syncwarp();
#pragma unroll
                for (int r0 = 0; r0 < 32; r0 += 32 / kLanes) {
                    const int r = r0 + sub;
                    if (r >= rows) continue;
                    const float* src = st + r * kEpiRow + col;
                    Out* dst = out + r * p.ldo + c0 + col;
                    if (sizeof(Out) == 4) {
                        *reinterpret_cast<float4*>(dst) = *reinterpret_cast<const float4*>(src);
                    } else {
                        const float4 u = *reinterpret_cast<const float4*>(src);
                        const float4 v = *reinterpret_cast<const float4*>(src + 4);
                        const __nv_bfloat162 o[4] = {__floats2bfloat162_rn(u.x, u.y), __floats2bfloat162_rn(u.z, u.w),
                                                     __floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
                        *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(o);
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
int launch(const Params& p, long long tiles, cudaStream_t s) {
    const int grid = (int)min(tiles, (long long)qbh::sm_count());
    k_mx_grad<kWeights, Out><<<grid, kThreads, smem_bytes(p.E), s>>>(p);
    return qbh::cuda_err(cudaGetLastError());
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

int mx_grad(const MxGrad& q, cudaStream_t s) {
    Params p{};
    // no rows: the map is not used, but its extent may not be 0
    if (!encode_rows(&p.a, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, q.R ? q.dy : q.out, q.R ? q.R : 1, q.N, q.lddy * 2, 64,
                     q.weights ? kC : kM))
        return QBMOE_ECUDA;
    p.dy = static_cast<const __nv_bfloat16*>(q.dy);
    p.lddy = q.lddy;
    p.codes = q.codes; p.scales = q.scales; p.offsets = q.offsets;
    p.out = q.out; p.ldo = q.ldo;
    p.R = q.R; p.E = q.E; p.N = q.N; p.K = q.K;
    p.m_tiles = (q.N + kM - 1) / kM;
    p.n_tiles = (q.K + kN - 1) / kN;
    p.status = mx_status();
    p.wait_limit = mx_wait_limit();
    p.stall = mx_stall();
    if (!q.weights) {
        const long long tiles = ((long long)(q.R / kM) + min(q.E, q.R)) * p.n_tiles;
        return launch<false, __nv_bfloat16>(p, tiles, s);
    }
    const long long tiles = (long long)q.E * p.m_tiles * p.n_tiles;
    return q.out_type == QBMOE_F32 ? launch<true, float>(p, tiles, s) : launch<true, __nv_bfloat16>(p, tiles, s);
}

}  // namespace qbh
