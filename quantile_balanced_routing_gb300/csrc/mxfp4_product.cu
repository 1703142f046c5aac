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
// 128-byte swizzle) and their scales.
//   warp 0     TMA producer (one lane)
//   warp 1     TMEM owner, MMA issuer (one lane): copies a stage's scales to
//              TMEM (tcgen05.cp, in order with the MMAs), 4 x K = 64 MMAs, one
//              commit that frees the stage
//   warp 2     the issuer's waiter (an mbarrier wait by the issuing thread
//              slows its MMA stream): waits, then releases it through a named barrier
//   warps 3, 4 scale loaders (even and odd stages): global -> registers one
//              stage ahead -> shared memory in the order tcgen05.cp wants
//   warps 5-8  epilogue: TMEM -> per-warp transpose in shared memory -> bf16
// Two accumulators alternate, so a tile's epilogue overlaps the next tile's
// main loop.  Every mbarrier wait is bounded: on expiry the kernel records
// QBMOE_ETIMEOUT, stops, lets its own copies and MMAs finish and frees TMEM.
#include "mxfp4.cuh"
#include "tc_ptx.cuh"

#include <cudaTypedefs.h>

#include <mutex>

namespace {

using namespace qb;

constexpr int kStageK = 256;                 // elements of K per stage (128 bytes of codes a row)
constexpr int kABytes = 128 * 128;           // weight codes of a stage
constexpr int kSfaBytes = 1024;              // weight scales of a stage: two 512-byte blocks (K = 128 each)
constexpr int kThreads = 288;
constexpr int kMmaWarp = 1, kWaitWarp = 2, kSfWarp = 3, kEpiWarp = 5;
constexpr int kHandoffBar = 1;
constexpr int kEpiRow = 36;                  // transpose row: 32 features, 4 words of padding
constexpr long long kDefaultWait = 1LL << 17;   // polls (<= 20 us each) before a wait expires
constexpr long long kDrainWait = 1LL << 12;

struct Params {
    CUtensorMap a, b;                        // codes of the weights [E N, K / 2] and of the rows [R, K / 2]
    const uint8_t* a_sc;                     // [E N, K / 32]
    const uint8_t* b_sc;                     // [R, K / 32]
    const int32_t* offsets;
    __nv_bfloat16* y;
    long long ldy;
    int R, E, N, K, nkb, m_total;
    int sf_bytes;                            // bytes of a scale load: 8 (K % 256 == 0), 4 (K % 128 == 0) or 1
    int weights_ready;                       // nothing enqueued just before this kernel wrote the weights or the offsets
    int* status;
    long long wait_limit;
    int stall;                               // test hook: withhold the first accumulator hand-off
};

template <int BN>
struct Shape {
    static constexpr int kBox = BN >= 32 ? 32 : 16;              // rows per TMA copy of B
    static constexpr int kNB = (BN + 127) / 128;                 // 128-row blocks of B's scales
    static constexpr int kBBytes = BN * 128;
    static constexpr int kSfbBytes = 2 * kNB * 512;
    static constexpr int kStage = kABytes + kBBytes + kSfaBytes + kSfbBytes;
    static constexpr int kSfCols = 2 * 4 + 2 * 4 * kNB;          // TMEM columns of a stage's scales
    static constexpr int kColsUsed = 2 * BN + 2 * kSfCols;       // two accumulators, two scale slots
    static constexpr uint32_t kCols = kColsUsed <= 64 ? 64 : kColsUsed <= 128 ? 128 : kColsUsed <= 256 ? 256 : 512;
    static_assert(kColsUsed <= 512, "TMEM columns");
    static constexpr int stages = BN == 16 ? 4 : BN == 64 ? 7 : BN == 128 ? 5 : 4;
    static constexpr int smem(int E) {
        return 1024 + stages * kStage + 4 * 16 * kEpiRow * 4 + (2 * (E + 1) + 64) * 4 + 256;
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
// 32 rows of 16 bytes (512 contiguous bytes) to 4 TMEM columns, the 32 lanes
// repeated in the four lane quarters.
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint32_t saddr) {
    // no swizzle; 8-row groups 128 bytes apart; descriptor version 1
    const uint64_t desc = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (1ull << 16) | (8ull << 32) | (1ull << 46);
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// The 8 scale bytes of one row and stage; bytes past the row's end are 0 (their codes are, too).
__device__ __forceinline__ uint2 load_scales(const uint8_t* row, int pitch, int kb, int bytes) {
    const uint8_t* p = row + kb * 8;
    if (bytes == 8) return __ldg(reinterpret_cast<const uint2*>(p));
    const int left = pitch - kb * 8;
    uint2 v = make_uint2(0, 0);
    if (bytes == 4) {
        v.x = __ldg(reinterpret_cast<const uint32_t*>(p));
        if (left > 4) v.y = __ldg(reinterpret_cast<const uint32_t*>(p) + 1);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = i < left ? __ldg(p + i) : 0u;
            if (i < 4) v.x |= b << (8 * i); else v.y |= b << (8 * (i - 4));
        }
    }
    return v;
}

template <int BN>
__global__ void __launch_bounds__(kThreads, BN == 16 ? 2 : 1) k_mx_product(const __grid_constant__ Params p) {
    using Sh = Shape<BN>;
    constexpr int S = Sh::stages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* a_ring = smem;
    uint8_t* b_ring = a_ring + S * kABytes;
    uint8_t* sfa_ring = b_ring + S * Sh::kBBytes;
    uint8_t* sfb_ring = sfa_ring + S * kSfaBytes;
    float* epi = reinterpret_cast<float*>(sfb_ring + S * Sh::kSfbBytes);    // [4][16][kEpiRow]
    uint64_t* full = reinterpret_cast<uint64_t*>(epi + 4 * 16 * kEpiRow);
    uint64_t* empty = full + S;
    uint64_t* accf = empty + S;
    uint64_t* acce = accf + 2;
    uint64_t* drain = acce + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* go_flag = reinterpret_cast<volatile int*>(tmem_slot + 2);   // [2]
    int* scratch = reinterpret_cast<int*>(tmem_slot + 4);                     // [kThreads / 32]
    Groups gr;
    gr.seg = scratch + 12;
    gr.toff = gr.seg + p.E + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long lim = p.wait_limit > 0 ? p.wait_limit : kDefaultWait;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            tc::mbar_init(&full[s], 2);      // the TMA producer and the stage's scale loader
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
        tc::prefetch_tmap(&p.b);
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(tmem_slot, Sh::kCols);
        tc::tmem_relinquish();
    }
    if (!p.weights_ready) pdl_wait();
    tc::tc_fence_before();
    load_groups<BN, kThreads>(gr, p.offsets, p.E, p.R, scratch);
    tc::tc_fence_after();
    const uint32_t tbase = *tmem_slot;
    const int n_tiles = gr.toff[p.E] * p.m_total;
    Walker<BN> w;
    w.start(gr, p.E, p.m_total, blockIdx.x);
    const int first = blockIdx.x, step = gridDim.x;

    if (warp == 0) {
        // ---------------------------------------------------------- TMA producer
        uint32_t issued = 0, last_par = 0;
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            bool rows_ready = !p.weights_ready;
            for (int t = first; t < n_tiles && !*abort_flag; t += step, w.next(gr, p.E, p.m_total, step)) {
                const int n_eff = (w.nrows + 15) & ~15;
                const int boxes = (n_eff + Sh::kBox - 1) / Sh::kBox;
                const int ya = w.g * p.N + w.m * 128;
                for (int kb = 0; kb < p.nkb; ++kb) {
                    if (!tc::mbar_wait(&empty[s], ph ^ 1u, lim)) {
                        set_status(p.status, QBMOE_ETIMEOUT);
                        *abort_flag = 1;
                        break;
                    }
                    tc::mbar_expect_tx(&full[s], kABytes + boxes * Sh::kBox * 128);
                    tc::tma_load_2d(a_ring + s * kABytes, &p.a, &full[s], kb * 128, ya);
                    if (!rows_ready) {   // the rows' codes come from the kernel before this one
                        pdl_wait();
                        rows_ready = true;
                    }
                    for (int i = 0; i < boxes; ++i)
                        tc::tma_load_2d(b_ring + s * Sh::kBBytes + i * Sh::kBox * 128, &p.b, &full[s], kb * 128,
                                        w.row0 + i * Sh::kBox);
                    issued |= 1u << s;
                    last_par = (last_par & ~(1u << s)) | (ph << s);
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
            }
        }
        __syncwarp();
        __syncthreads();
        if (lane == 0 && *abort_flag)   // every copy has landed before shared memory is released
            for (int s = 0; s < S; ++s)
                if ((issued >> s) & 1u) tc::mbar_wait(&full[s], (last_par >> s) & 1u, kDrainWait);
    } else if (warp == kSfWarp || warp == kSfWarp + 1) {
        // ---------------------------------------------------------- scale loaders
        // Loader v takes the stages it = v, v + 2, ... of the CTA's sequence of
        // (tile, K block) pairs and has the next one's bytes in registers while
        // it waits for a slot.
        constexpr int kBJ = BN / 32 + (BN % 32 ? 1 : 0);
        const int v = warp - kSfWarp, pitch = p.K / 32;
        const long long last_a = (long long)p.E * p.N - 1;
        uint2 ra[4], rb[kBJ];
        auto fetch = [&](int kb) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const long long row = min((long long)w.g * p.N + w.m * 128 + lane + 32 * j, last_a);
                ra[j] = load_scales(p.a_sc + row * pitch, pitch, kb, p.sf_bytes);
            }
#pragma unroll
            for (int j = 0; j < kBJ; ++j) {
                const int r = min(w.row0 + lane + 32 * j, p.R - 1);
                rb[j] = 32 * j < w.nrows ? load_scales(p.b_sc + (long long)r * pitch, pitch, kb, p.sf_bytes)
                                         : make_uint2(0, 0);
            }
        };
        if (p.weights_ready) pdl_wait();
        int t = first, kb = v;
        bool have = t < n_tiles;
        auto settle = [&] {   // kb may run past its tile: into the next ones
            while (have && kb >= p.nkb) {
                kb -= p.nkb;
                t += step;
                have = t < n_tiles && w.next(gr, p.E, p.m_total, step);
            }
        };
        settle();
        if (have) fetch(kb);
        int s = v;
        uint32_t ph = 0;
        while (s >= S) { s -= S; ph ^= 1u; }
        while (have) {
            int ok = 1;
            if (lane == 0) {
                ok = !*abort_flag && tc::mbar_wait(&empty[s], ph ^ 1u, lim);
                if (!ok) {
                    set_status(p.status, *abort_flag ? 0 : QBMOE_ETIMEOUT);
                    *abort_flag = 1;
                }
            }
            if (!__shfl_sync(0xffffffffu, ok, 0)) break;
            uint4* A = reinterpret_cast<uint4*>(sfa_ring + s * kSfaBytes);
            A[lane] = make_uint4(ra[0].x, ra[1].x, ra[2].x, ra[3].x);
            A[32 + lane] = make_uint4(ra[0].y, ra[1].y, ra[2].y, ra[3].y);
            uint4* B = reinterpret_cast<uint4*>(sfb_ring + s * Sh::kSfbBytes);
#pragma unroll
            for (int nb = 0; nb < Sh::kNB; ++nb) {
                uint32_t x[4] = {}, y[4] = {};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (4 * nb + j < kBJ) x[j] = rb[4 * nb + j].x, y[j] = rb[4 * nb + j].y;
                B[nb * 32 + lane] = make_uint4(x[0], x[1], x[2], x[3]);
                B[(Sh::kNB + nb) * 32 + lane] = make_uint4(y[0], y[1], y[2], y[3]);
            }
            kb += 2;
            settle();
            if (have) fetch(kb);
            tc::fence_proxy_async_smem();   // generic-proxy writes -> tcgen05.cp reads
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&full[s]);
            s += 2;
            if (s >= S) { s -= S; ph ^= 1u; }
        }
        __syncthreads();
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------- MMA issuer
        int s = 0, ab = 0, h = 0, sb = 0;
        const uint64_t a0 = tc::desc_sw128(tc::smem_u32(a_ring)), b0 = tc::desc_sw128(tc::smem_u32(b_ring));
        const uint32_t sfa0 = tc::smem_u32(sfa_ring), sfb0 = tc::smem_u32(sfb_ring);
        for (int t = first; t < n_tiles; t += step, w.next(gr, p.E, p.m_total, step)) {
            const uint32_t n_eff = (w.nrows + 15) & ~15;
            const uint32_t id[2] = {idesc_mxf4(n_eff, 0), idesc_mxf4(n_eff, 2)};
            const int nb = n_eff > 128 ? 2 : 1;
            tc::named_bar_sync(kHandoffBar, 64);   // the accumulator is free (or stop)
            const bool go = go_flag[h & 1] != 0;
            ++h;
            if (!go) break;
            const uint32_t d = tbase + ab * BN;
            for (int kb = 0; kb < p.nkb; ++kb) {
                tc::named_bar_sync(kHandoffBar, 64);   // stage s has landed
                if (lane == 0) {
                    tc::tc_fence_after();
                    const uint32_t ca = tbase + 2 * BN + sb * Sh::kSfCols, cb = ca + 8;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        cp_scales(ca + 4 * c, sfa0 + s * kSfaBytes + 512 * c);
                        for (int i = 0; i < nb; ++i)
                            cp_scales(cb + 4 * (Sh::kNB * c + i), sfb0 + s * Sh::kSfbBytes + 512 * (Sh::kNB * c + i));
                    }
                    const uint64_t ad = a0 + (uint64_t)(s * (kABytes >> 4)), bd = b0 + (uint64_t)(s * (Sh::kBBytes >> 4));
                    const int left = p.K - kb * kStageK;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        if (kk * 64 < left)
                            mma_mxf4(d, ad + 2 * kk, bd + 2 * kk, id[kk & 1], ca + 4 * (kk >> 1),
                                     cb + 4 * Sh::kNB * (kk >> 1), (kb | kk) != 0);
                    tc::tc_commit(&empty[s]);
                }
                __syncwarp();
                sb ^= 1;
                if (++s == S) s = 0;
            }
            if (lane == 0 && !(p.stall && t == first)) tc::tc_commit(&accf[ab]);
            __syncwarp();
            ab ^= 1;
        }
        if (lane == 0) {   // every MMA and copy of this thread is done before TMEM is freed
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
                if (!dead && !tc::mbar_wait(&acce[ab], aph ^ 1u, lim)) {
                    set_status(p.status, QBMOE_ETIMEOUT);
                    *abort_flag = 1;
                    dead = true;
                }
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
                    if (!dead && !tc::mbar_wait(&full[s], ph, lim)) {
                        set_status(p.status, QBMOE_ETIMEOUT);
                        *abort_flag = 1;
                        dead = true;
                    }
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
        // Lane q * 32 + lane of an accumulator holds weight row m * 128 + 32 q +
        // lane; a warp turns 16 rows' worth of its 32 features around in its own
        // piece of shared memory and stores 64 bytes a row.
        const int q = warp & 3;
        float* st = epi + q * 16 * kEpiRow;
        int ab = 0;
        uint32_t fph = 0;
        for (int t = first; t < n_tiles; t += step, w.next(gr, p.E, p.m_total, step)) {
            int ok = 1;
            if (lane == 0) {
                ok = tc::mbar_wait(&accf[ab], fph, lim);
                if (!ok) {
                    set_status(p.status, QBMOE_ETIMEOUT);
                    *abort_flag = 1;
                }
            }
            if (!__shfl_sync(0xffffffffu, ok, 0)) break;
            tc::tc_fence_after();
            const int j = lane >> 1, half = lane & 1;
            const int f = w.m * 128 + 32 * q + 16 * half;
            __nv_bfloat16* out = p.y + (long long)(w.row0 + j) * p.ldy + f;
            for (int c0 = 0; c0 < w.nrows; c0 += 16) {
                float v[16];
                tc::tmem_ld16(tbase + ab * BN + (static_cast<uint32_t>(32 * q) << 16) + c0, v);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 16; ++i) st[i * kEpiRow + lane] = v[i];
                __syncwarp();
                if (c0 + j < w.nrows) {
                    const float4* src = reinterpret_cast<const float4*>(st + j * kEpiRow + 16 * half);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const float4 a = src[2 * g], b = src[2 * g + 1];
                        const __nv_bfloat162 o[4] = {__floats2bfloat162_rn(a.x, a.y), __floats2bfloat162_rn(a.z, a.w),
                                                     __floats2bfloat162_rn(b.x, b.y), __floats2bfloat162_rn(b.z, b.w)};
                        if (f + 8 * g < p.N)
                            *reinterpret_cast<uint4*>(out + (long long)c0 * p.ldy + 8 * g) =
                                *reinterpret_cast<const uint4*>(o);
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
        tc::tmem_dealloc(tbase, Sh::kCols);
    }
    pdl_wait();   // also a CTA without tiles ends after the kernel before this one
}

constexpr int kMaxDevices = 64;
__device__ int g_status;
int* g_status_ptr[kMaxDevices] = {};
int g_sms[kMaxDevices] = {};
long long g_wait_limit = 0;
int g_stall = 0;

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
    if (!qbh::encode_rows(&p.b, CU_TENSOR_MAP_DATA_TYPE_UINT8, q.x_codes, q.R, q.K / 2, q.K / 2, 128, Shape<BN>::kBox))
        return QBMOE_ECUDA;
    // row tiles of all experts: at most one ragged tile for each that has rows
    const long long tiles = ((long long)(q.R / BN) + min(q.E, q.R)) * p.m_total;
    const int grid = (int)min(tiles, (long long)qbh::sm_count() * (BN == 16 ? 2 : 1));
    const size_t smem = Shape<BN>::smem(q.E);
    if (q.raw) {
        // the product may set itself up, and load weights, while its rows are quantised
        const int rc = qbh::mx_quantize(q.R, q.K, q.raw_type, q.raw, q.raw_ld, q.x_codes, q.x_scales, nullptr, s);
        if (rc) return rc;
        return qbh::launch_pdl(k_mx_product<BN>, dim3(grid), dim3(kThreads), smem, s, p);
    }
    k_mx_product<BN><<<grid, kThreads, smem, s>>>(p);
    return qbh::cuda_err(cudaGetLastError());
}

}  // namespace

namespace qbh {

int mx_product_init() {
    const int dev = current_device();
    if (dev < 0) return QBMOE_ECUDA;
    void* f = nullptr;
    int rc = cuda_err(cudaGetSymbolAddress(&f, g_status));
    if (!rc) rc = cuda_err(cudaDeviceGetAttribute(&g_sms[dev], cudaDevAttrMultiProcessorCount, dev));
    if (!rc) rc = set_attributes<16>();
    if (!rc) rc = set_attributes<64>();
    if (!rc) rc = set_attributes<128>();
    if (!rc) rc = set_attributes<224>();
    if (!rc) g_status_ptr[dev] = static_cast<int*>(f);
    return rc;
}

int* mx_status() {
    const int dev = current_device();
    return dev < 0 ? nullptr : g_status_ptr[dev];
}
int mx_status_take() {
    int* p = mx_status();
    if (!p) return QBMOE_OK;   // no call has run on this device
    int v = 0;
    if (cudaMemcpy(&v, p, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return QBMOE_ECUDA;
    if (v != 0 && cudaMemset(p, 0, 4) != cudaSuccess) return QBMOE_ECUDA;
    return v;
}
long long mx_wait_limit() { return g_wait_limit; }
void mx_set_wait_limit(long long polls) { g_wait_limit = polls > 0 ? polls : 0; }
int mx_stall() { return g_stall; }
void mx_set_stall(int on) { g_stall = on; }
int sm_count() {
    const int dev = current_device();
    return dev < 0 || g_sms[dev] < 1 ? 1 : g_sms[dev];
}

bool encode_rows(CUtensorMap* m, CUtensorMapDataType type, const void* base, long long rows, long long cols,
                 long long ld_bytes, int box_cols, int box_rows) {
    const auto encode = encoder();
    if (!encode) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld_bytes};
    cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    cuuint32_t es[2] = {1, 1};
    return encode(m, type, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int mx_product(const MxProduct& q, cudaStream_t s) {
    Params p{};
    if (!encode_rows(&p.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, q.w_codes, (long long)q.E * q.N, q.K / 2, q.K / 2, 128, 128))
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
    p.status = mx_status();
    p.wait_limit = g_wait_limit;
    p.stall = g_stall;
    // Row tile: the smallest that holds an average expert's rows.
    const int avg = (q.R + q.E - 1) / q.E;
    if (avg <= 16) return launch<16>(q, p, s);
    if (avg <= 64) return launch<64>(q, p, s);
    if (avg <= 128) return launch<128>(q, p, s);
    return launch<224>(q, p, s);
}

}  // namespace qbh
