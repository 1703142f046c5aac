/*
 * qbmoe — Stable LatentMoE forward with Quantile Balancing on one GB300 (sm_103a).
 *
 * C ABI.  Plain pointers and sizes only.  "Device" pointers are CUDA device
 * (or managed) memory on the current device; "host" pointers are ordinary
 * host memory.  Every call that takes a stream is asynchronous and
 * stream-ordered on it (NULL = the legacy default stream); nothing here
 * synchronises the host except qbmoe_status and the functions documented as
 * synchronous.
 *
 * Errors.  Every call checks its arguments, encodes every tensor map and
 * sets up the device (kernel attributes, once per device) before its first
 * launch; a negative code from any of those steps means nothing was
 * launched and no output was touched.  Only QBMOE_ECUDA can also come from a
 * launch itself (the CUDA runtime refusing a launch or a copy); then the
 * launches that preceded it in the same call stay enqueued and the call's
 * outputs may be partly written.  Failures inside kernels are reported
 * later, by qbmoe_status.
 *
 * Sources, by page title and section:
 *   [K3-width]  "Kimi K3 模型结构（5）：宽度维度，Stable LatentMoE" (xhh.club),
 *               its 延伸解读 (extended reading) sections and its Q&A.
 *   [K3-explainer]  "KIMI K3" LatentMoE explainer (dimsnsums.com),
 *               "Why does the router need three moves?".
 */
#ifndef QBMOE_H
#define QBMOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Compatible with cudaStream_t. */
typedef struct CUstream_st* qbmoe_stream_t;

typedef enum {
    QBMOE_OK = 0,
    QBMOE_EINVAL = -1,     /* bad size, null or misaligned pointer, unsupported option */
    QBMOE_ENOMEM = -2,     /* device allocation failed (qbmoe_create, qbmoe_pack_weights) */
    QBMOE_ECUDA = -3,      /* a CUDA runtime/driver call or a launch failed */
    QBMOE_EARCH = -4,      /* current device is not compute capability 10.3 */
    QBMOE_EWORKSPACE = -5, /* caller workspace too small / ctx built for fewer tokens */
    QBMOE_ETIMEOUT = -6,   /* a kernel's bounded wait expired (reported by qbmoe_status) */
    QBMOE_EDEVICE = -7     /* a kernel's own check failed (reported by qbmoe_status) */
} qbmoe_status_t;

/* Storage types. */
enum { QBMOE_F32 = 0, QBMOE_BF16 = 1, QBMOE_MXFP4 = 2 /* moe_mxfp4_matmul's rows only */,
       QBMOE_MXFP8 = 3 /* rows of moe_mxfp4_matvec and moe_mxfp4_experts only */ };
/* Routed-expert weight formats. */
enum { QBMOE_W_F32 = 0, QBMOE_W_BF16 = 1, QBMOE_W_MXFP4 = 2 };
/* QB sweep forms: every expert from the same biases (the default, one
 * exchange of per-expert quantiles per sweep), or cyclic coordinate descent
 * (each expert's step sees the latest biases; moe_route_qb_gs). */
enum { QBMOE_QB_JACOBI = 0, QBMOE_QB_GAUSS_SEIDEL = 1 };

/* Limits of this build. */
#define QBMOE_MAX_EXPERTS 1024
#define QBMOE_MAX_TOPK 32
/* Tokens, sequences or rows of a router-training or MXFP4 product call: 2^31 - 2^24, so
 * that sizes rounded up to tiles, and row and tile counts added, stay in 32 bits. */
#define QBMOE_MAX_ROWS 2130706432

/*
 * Scores.  s = sigmoid(logit) is an exactly specified fp32 result: clamp the
 * logit to [-80, 80], y = -x, j = rint(y*0x1.715476p+0),
 * r = (y - j*0x1.62e4p-1) - j*0x1.7f7d1cp-20, p = degree-7 Taylor series of
 * e^r in Horner form (coefficients 1/5040, 1/720, 1/120, 1/24, 1/6 rounded to
 * fp32, then 1/2, 1, 1), e = p*2^j, s = 1/(1+e); every step one IEEE fp32
 * operation, no fused multiply-add.  ([K3-width] Q&A on routing: sigmoid
 * router on the full-width input.)
 */

/*
 * ---------------------------------------------------------------------------
 * moe_route_qb — router scores, Quantile Balancing, biased top-k.
 *
 * [K3-width] Q&A on Quantile Balancing: each expert's bias is the (1 - k/n)
 * quantile over tokens of its margin, minus a common offset, so that every
 * expert admits its target load T*k/n; 延伸解读 "QB vs DeepSeek-V3": one
 * exact coordinate-descent step on the balanced-assignment dual.  Q&A on
 * routing: top-k on score + bias, mixture weights = raw scores renormalised
 * over the chosen k, bias frozen at inference (qb_sweeps = 0).
 *
 * Per sweep (Jacobi: every expert from the same bias b):
 *   v = fl(s + b); per token the experts ranked by (v desc, index asc);
 *   tau[t][j] = the (k+1)-th ranked v if j is in the token's top k, else the
 *   k-th; m[t][j] = fl(s - tau) (-0 -> +0);
 *   r_j = floor(T*k/n) + (j < T*k mod n);  M = m[.][j] sorted descending;
 *   q_j = fl(fl(M_r + M_{r+1}) * 0.5)  (r=0: fl(M_1 + 1); r>=T: fl(M_T - 1));
 *   b'_j = -q_j;  c = fl(S / n), S = pairwise tree sum of b' padded with +0
 *   to 2^ceil(log2 n); b = fl(b' - c).
 * Final: idx[t] = top k of fl(s + b) in rank order; w[t][i] =
 * fl(s[idx_i] / sum), sum accumulated in rank order in fp32;
 * loads[j] = number of routes to j.
 *
 * T >= 1, 2 <= n <= QBMOE_MAX_EXPERTS, 1 <= k < n, k <= QBMOE_MAX_TOPK,
 * qb_sweeps >= 0.
 * logits   [T, n] fp32 device, row-major, pre-sigmoid.
 * bias_in  [n] fp32 device (NULL = zeros).  bias_out [n] fp32 device; may
 *          equal bias_in.
 * scores   [T, n] fp32 device out.  topk_idx [T, k] int32, topk_w [T, k]
 *          fp32, loads [n] int32 device out.
 * workspace: device, >= qbmoe_route_workspace_bytes(T, n, k) bytes, 256-byte
 *          aligned; owned by the caller; contents are scratch.
 * All device pointers 16-byte aligned.  Results are bit-reproducible.
 * Returns QBMOE_OK after enqueueing, or a negative code (see Errors above).
 */
size_t qbmoe_route_workspace_bytes(int T, int n, int k);
int moe_route_qb(int T, int n, int k, int qb_sweeps,
                 const float* logits, const float* bias_in, float* bias_out,
                 float* scores, int32_t* topk_idx, float* topk_w, int32_t* loads,
                 void* workspace, size_t workspace_bytes, qbmoe_stream_t stream);

/*
 * moe_route_qb_gs — Quantile Balancing by cyclic coordinate descent.
 *
 * [K3-width] 延伸解读 "QB vs DeepSeek-V3": QB solves the balanced-assignment
 * dual by coordinate descent, jumping to the exact coordinate minimiser.
 * This is the literal cyclic form: within a sweep the experts are updated in
 * order j = 0..n-1, each step computing expert j's margins under the latest
 * biases (tau[t][j] = k-th best fl(s + b) among the other experts) and
 * setting b_j = -midpoint of its r_j-th and (r_j+1)-th largest margins, as in
 * moe_route_qb; after the sweep the common offset is subtracted.  Repeated
 * sweeps never raise the dual; once every expert's load equals its target
 * the assignment is optimal for the balanced problem.
 *
 * max_sweeps >= 0 sweeps are run; with stop_when_balanced != 0 the sweeps
 * stop (on the device) after the first sweep whose loads equal the targets.
 * sweeps_done: device int32 or NULL, receives the number of sweeps run.
 * Other arguments as moe_route_qb; workspace >= qbmoe_route_gs_workspace_bytes.
 * Cost: about 2n + 5 kernel launches per sweep (a quality mode for balancing,
 * not the layer's hot path, which uses the one-pass Jacobi sweep).
 */
size_t qbmoe_route_gs_workspace_bytes(int T, int n, int k);
int moe_route_qb_gs(int T, int n, int k, int max_sweeps, int stop_when_balanced,
                    const float* logits, const float* bias_in, float* bias_out,
                    float* scores, int32_t* topk_idx, float* topk_w, int32_t* loads,
                    int32_t* sweeps_done, void* workspace, size_t workspace_bytes,
                    qbmoe_stream_t stream);

/*
 * moe_route_signsgd — DeepSeek-V3's fixed-step sign rule, the comparator of
 * Quantile Balancing.
 *
 * [K3-width] 延伸解读 "QB vs DeepSeek-V3": DeepSeek-V3 moves each expert's
 * bias by a fixed, hand-tuned step along a sign; that rule is SignSGD on the
 * same dual that QB minimises exactly.  From b = bias_in (NULL = zeros),
 * `steps` times: loads under the biased top-k of b, then
 *   b_j = fl(b_j - gamma) if load_j > r_j;  fl(b_j + gamma) if load_j < r_j;
 *   unchanged if load_j = r_j  (r_j as in moe_route_qb, no common offset).
 * Then the final routing on b as in moe_route_qb; bias_out = b.
 * steps >= 0, 0 < gamma < inf; other arguments as moe_route_qb, workspace
 * >= qbmoe_route_signsgd_workspace_bytes(T, n, k).  Bit-reproducible.
 */
size_t qbmoe_route_signsgd_workspace_bytes(int T, int n, int k);
int moe_route_signsgd(int T, int n, int k, int steps, float gamma,
                      const float* logits, const float* bias_in, float* bias_out,
                      float* scores, int32_t* topk_idx, float* topk_w, int32_t* loads,
                      void* workspace, size_t workspace_bytes, qbmoe_stream_t stream);

/*
 * Token-sharded Quantile Balancing with a histogram exchange.
 *
 * [K3-width] Q&A on Quantile Balancing: the quantiles are formed from
 * histogram estimates so that the communication stays cheap.  A batch of
 * T_total tokens is split into shards (on one or several devices); no shard
 * sees another's margins.  Each expert's coordinate step needs the r_j-th
 * and (r_j+1)-th largest margin over the whole batch (moe_route_qb).  Four
 * passes each exchange, per expert and per tracked rank, the 256-bin
 * histogram of one 8-bit digit of the margins' order keys among the keys
 * that match the digits fixed so far (n * 2 * 256 int32 per pass, against
 * T_total * n margins), and refine the estimate until both order
 * statistics are exact.  The bias is then bit-identical to moe_route_qb's
 * one-sweep bias of the whole batch, and each shard routes its tokens with
 * moe_route_qb(qb_sweeps = 0, bias_in = that bias).
 *
 * Per sweep:
 *   moe_qb_hist_init(T_total, n, k, state, hist)          targets, zeroed hist
 *   moe_qb_shard_margins(shard)                          each local shard
 *   for pass = 0..3:
 *     moe_qb_shard_hist(shard, pass, state, ws, hist)    each local shard ADDS
 *                                                        its counts into hist
 *     (the caller sums hist over devices: an all-reduce)
 *     moe_qb_hist_advance(n, pass, hist, state)          fixes the digit and
 *                                                        zeroes hist
 *   moe_qb_hist_bias(n, state, bias)                      b' and common offset
 *
 * state: device, qbmoe_qb_hist_state_bytes(n), caller-owned, one per device
 * (every device holds the same state after each advance).  hist: device
 * int32 [n][2][256] (qbmoe_qb_hist_bytes(n)).  Shard workspace: device,
 * qbmoe_qb_shard_workspace_bytes(T_shard, n, k), 256-byte aligned; holds the
 * shard's margins [n, T_shard] from moe_qb_shard_margins until its last
 * moe_qb_shard_hist.  moe_qb_shard_margins: logits [T_shard, n] fp32 in,
 * scores [T_shard, n] fp32 out, bias_in [n] or NULL (zeros) - the bias the
 * sweep starts from, the same on every shard.  T_total * k < 2^31.
 */
size_t qbmoe_qb_hist_state_bytes(int n);
size_t qbmoe_qb_hist_bytes(int n);
size_t qbmoe_qb_shard_workspace_bytes(int T_shard, int n, int k);
int moe_qb_hist_init(int T_total, int n, int k, void* state, int32_t* hist, qbmoe_stream_t stream);
int moe_qb_shard_margins(int T_shard, int n, int k, const float* logits, const float* bias_in, float* scores,
                         void* workspace, size_t workspace_bytes, qbmoe_stream_t stream);
int moe_qb_shard_hist(int T_shard, int n, int pass, const void* state, const void* workspace, int32_t* hist,
                      qbmoe_stream_t stream);
int moe_qb_hist_advance(int n, int pass, int32_t* hist, void* state, qbmoe_stream_t stream);
int moe_qb_hist_bias(int n, const void* state, float* bias_out, qbmoe_stream_t stream);

/*
 * moe_route_qb_noalloc — moe_route_qb for callers that cannot allocate.
 *
 * The pages have no counterpart: this is a deployment variant of the router
 * above with identical results, for callers that cannot hand it a workspace
 * because they may not allocate device memory where they route (a serving
 * path whose device memory is planned up front and may not grow, or a
 * plug-in that only receives its inputs and outputs from a host program
 * that owns all memory).  Arguments are those
 * of moe_route_qb without the workspace.  The scratch lives in one fixed
 * device array of qbmoe_route_noalloc_max_bytes() bytes (32 MiB) that every
 * GPU which loads the library keeps until the process exits; sizes whose
 * scratch (qbmoe_route_workspace_bytes(T, n, k)) exceeds it are refused with
 * QBMOE_EWORKSPACE before anything is launched.  The call makes no cudaMalloc
 * or cudaFree and calls no allocating library routine.
 *
 * The first call on a device looks up the array's device address on that
 * device (cudaGetSymbolAddress) and sets the library's kernel attributes
 * there; make that first call before any stream capture.  All calls share
 * the one array, so calls that may overlap on the GPU (different streams, or
 * different host threads on one device) race and must be serialised by the
 * caller.  Nothing needs to start at zero: every
 * scratch region is written before it is read.
 */
size_t qbmoe_route_noalloc_max_bytes(void);
int moe_route_qb_noalloc(int T, int n, int k, int qb_sweeps,
                         const float* logits, const float* bias_in, float* bias_out,
                         float* scores, int32_t* topk_idx, float* topk_w, int32_t* loads,
                         qbmoe_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Router training: balance loss, per-expert counts and the logits' gradient.
 *
 * A batch of T tokens is cut into S sequences, seq_offsets [S + 1] (int32
 * device, non-decreasing from 0 to T; NULL = one sequence of all T tokens).
 * token_mask [T] (device bytes, 0 = padding, not counted; NULL = all valid).
 * idx [T, k] int32 device: the experts each token was routed to, distinct; an
 * entry outside [0, n) stands for no route.  logits [T, n], row stride ld >= n
 * elements, QBMOE_F32 or QBMOE_BF16 (logit_dtype).
 *
 * With s = sigmoid(logit clamped to [-80, 80]) (the router's score), the share
 * p[t][j] = s[t][j] / sum_l s[t][l], and over the valid tokens V_q of sequence q
 * (T_q of them):
 *   counts[q][j] = routes of V_q to expert j
 *   probs[q][j]  = mean over V_q of p[t][j]
 *   loss[q]      = n / (k T_q) * sum_j counts[q][j] probs[q][j]
 * loss[q] is 1 when every expert has the same count or the same mean share;
 * a sequence without valid tokens has zeros throughout.  (The auxiliary loss
 * of sigmoid routers, per sequence; the caller weighs and sums loss[q].)
 *
 * moe_balance_loss writes loss [S] fp32, counts [S, n] int32, probs [S, n]
 * fp32 and tokens [S] int32 (T_q).  workspace: device, 256-byte aligned,
 * >= qbmoe_balance_workspace_bytes(T, n, S) bytes.  Sums are fp32 in a fixed
 * order: bit-reproducible.
 *
 * moe_router_backward writes dlogits [T, n] (row stride ldg, of logit_dtype),
 * the gradient of
 *   sum_t sum_i dw[t][i] w[t][i] + sum_q dloss[q] loss[q]
 * where w[t][i] = s[t][idx_i] / sum_l s[t][idx_l] are the mixture weights and
 * the routes (idx, counts) are constants.  dw [T, k] fp32 or NULL (no such
 * term); dloss [S] fp32 with counts and tokens as moe_balance_loss wrote them,
 * or all three NULL.  Padding tokens, and logits outside [-80, 80], get 0.
 * dlogits may equal logits (same stride).
 *
 * 1 <= T <= QBMOE_MAX_ROWS, 2 <= n <= QBMOE_MAX_EXPERTS, 1 <= k <= min(n, QBMOE_MAX_TOPK),
 * 1 <= S <= QBMOE_MAX_ROWS.  Device pointers are aligned to their element type only: rows of a
 * 16-byte-aligned base and stride are read as vectors.
 */
size_t qbmoe_balance_workspace_bytes(int T, int n, int S);
int moe_balance_loss(int T, int n, int k, int S, int logit_dtype, const void* logits, long long ld,
                     const int32_t* idx, const int32_t* seq_offsets, const uint8_t* token_mask,
                     float* loss, int32_t* counts, float* probs, int32_t* tokens,
                     void* workspace, size_t workspace_bytes, qbmoe_stream_t stream);
int moe_router_backward(int T, int n, int k, int S, int logit_dtype, const void* logits, long long ld,
                        const int32_t* idx, const int32_t* seq_offsets, const uint8_t* token_mask,
                        const float* dw, const float* dloss, const int32_t* counts, const int32_t* tokens,
                        void* dlogits, long long ldg, qbmoe_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * MXFP4 tensors: quantisation, product and its gradients.
 *
 * An MXFP4 tensor [rows, K] is codes [rows, K/2] u8 (E2M1, element 2i in the
 * low nibble) and scales [rows, K/32] u8 (E8M0: 2^(byte - 127)), both
 * contiguous: the layout of the layer's routed-expert weights (qbmoe_weights).
 * K is a multiple of 32.
 *
 * moe_mxfp4_quantize: x [rows, K] (QBMOE_F32 or QBMOE_BF16, row stride ldx
 * elements) to codes and scales.  Per 32 elements, e = floor(log2 max|x|) - 2
 * (at least -127; -127 for a block of zeros), code = x * 2^-e rounded to
 * nearest, ties to even, magnitudes above 6 to 6; the sign of zero is kept.  A block that
 * holds an infinity or a NaN gets the scale byte 0xFF (NaN) and zero codes.
 * values (NULL if not wanted): [rows, K] contiguous, of x's type, what the codes
 * stand for, exact in either type (NaN throughout a 0xFF block).
 * x, codes and values 16-byte aligned, ldx * element size a multiple of 16, rows * K at
 * most 2^40.
 *
 * Grouped rows: R rows in expert order, offsets [E + 1] int32 device,
 * non-decreasing from 0 to R: rows offsets[e] .. offsets[e+1] - 1 belong to
 * expert e (an expert may have none).  offsets NULL: E = 1, all rows.
 * Rows that no expert owns are not written.  0 <= R <= QBMOE_MAX_ROWS, 1 <= E <=
 * QBMOE_MAX_EXPERTS, N a multiple of 8.
 *
 * moe_mxfp4_matmul:  y[r][f] = sum_k x[r][k] w[e(r)][f][k], x and w MXFP4
 *   ([R, K] and [E, N, K]), y [R, N] bf16, row stride ldy elements.  x_type
 *   QBMOE_MXFP4: x the codes, x_scales the scales, ldx = K.  x_type QBMOE_F32
 *   or QBMOE_BF16: x [R, K] of that type, row stride ldx elements, quantised
 *   into the workspace first as moe_mxfp4_quantize does; x_scales is not used.
 *   workspace: device, 256-byte aligned, >= qbmoe_mxfp4_workspace_bytes(R, K)
 *   bytes; not used, and may be NULL, when x is MXFP4.
 * moe_mxfp4_dgrad:   dx[r][k] = sum_f dy[r][f] w[e(r)][f][k], dy [R, N] bf16
 *   (row stride lddy), dx [R, K] bf16 (row stride lddx).
 * moe_mxfp4_wgrad:   dw[e][f][k] = sum over e's rows of dy[r][f] x[r][k],
 *   dw [E, N, K] contiguous, QBMOE_F32 or QBMOE_BF16; zeros for an expert
 *   without rows.  workspace: device, 256-byte aligned, >=
 *   qbmoe_mxfp4_wgrad_workspace_bytes(R, E, N, K) bytes (0, and NULL allowed,
 *   unless the matrices are few and small).
 * The gradients are those of the product for the values x and w stand for; a
 * trainer that quantises its own activations and weights passes them straight
 * through the rounding.  A value above bf16's largest (scale bytes 253 and 254 with
 * codes from 4 or 2 on; the quantiser makes none) counts as infinite in them.
 * Products are exact.  Sums are the tensor cores' fp32 accumulation, which drops low
 * bits (7e-6 of the norm over 40000 terms).  An fp32 weight gradient is therefore
 * accumulated 4096 rows at a time, and the segments, like the parts that a workspace
 * is for, added in fp32 (2e-7); a bf16 one only where it is cut into parts.
 * Each output is rounded to its type once.  All pointers 16-byte aligned, strides multiples of 8 elements and at
 * most 2^27, N and K at most 2^24, E N below 2^31.
 * A bounded wait that expires is reported by qbmoe_status(NULL, stream).
 */
int moe_mxfp4_quantize(long long rows, int K, int x_type, const void* x, long long ldx, uint8_t* codes,
                       uint8_t* scales, void* values, qbmoe_stream_t stream);
size_t qbmoe_mxfp4_workspace_bytes(int R, int K);
int moe_mxfp4_matmul(int R, int E, int N, int K, int x_type, const void* x, long long ldx, const uint8_t* x_scales,
                     const uint8_t* w_codes, const uint8_t* w_scales, const int32_t* offsets, void* y, long long ldy,
                     void* workspace, size_t workspace_bytes, qbmoe_stream_t stream);
int moe_mxfp4_dgrad(int R, int E, int N, int K, const void* dy, long long lddy, const uint8_t* w_codes,
                    const uint8_t* w_scales, const int32_t* offsets, void* dx, long long lddx,
                    qbmoe_stream_t stream);
size_t qbmoe_mxfp4_wgrad_workspace_bytes(int R, int E, int N, int K);
int moe_mxfp4_wgrad(int R, int E, int N, int K, const void* dy, long long lddy, const uint8_t* x_codes,
                    const uint8_t* x_scales, const int32_t* offsets, int dw_dtype, void* dw,
                    void* workspace, size_t workspace_bytes, qbmoe_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * The norm in front of a layer: the residual's addition, RMS norm of the sum,
 * rows in 8 bits, and the gradient.
 *
 * An MXFP8 tensor [rows, K] is codes [rows, K] u8 (E4M3) and scales [rows, K/32]
 * u8 (E8M0: 2^(byte - 127)), both contiguous; K is a multiple of 32.
 *
 * moe_add_rmsnorm, per row of H elements:
 *   total = x + residual, one fp32 sum rounded to the residual's type
 *   r = 1 / sqrt(sum_j total_j^2 / H + eps),  n_j = (total_j r) gamma_j
 * x [T, H] of x_type, residual and total [T, H] of res_type (each QBMOE_F32 or
 * QBMOE_BF16; total may be the residual, or x where types and strides agree).
 * residual and total NULL: the norm of x itself.  gamma [H] fp32.
 * codes NULL: y [T, H] of x_type takes n rounded once.  Else codes and scales
 * take n in MXFP8 (H a multiple of 32): per 32 elements e = floor(log2 max|n|) - 7
 * (at least -127; -127 for a block of zeros), code = n 2^-e in E4M3, rounded to
 * nearest, ties to even.  Scaled magnitudes are below 256, so that none saturates.
 * A block that holds an infinity or a NaN gets the scale byte 0xFF (NaN) and zero
 * codes.  y, which may then be NULL, takes the values that the codes stand for, in
 * QBMOE_BF16 (exact down to 2^-133; NaN throughout a 0xFF block).
 *
 * moe_add_rmsnorm_backward: for dn, the gradient of n (straight through the
 * rounding), with total as moe_add_rmsnorm wrote it (x where there is no
 * residual) and r of it formed anew:
 *   dx = dtotal + r (g - total r^2 mean_j(g total)),  g = dn gamma
 *   dgamma_j = sum_t dn total r
 * dx, of total_type, is the gradient of x and of the residual alike; dtotal, of
 * total_type, is the total's own gradient (NULL: none).  dn of dn_type.  dx may be dtotal (same
 * stride), or dn where the types and strides agree.  dgamma [H] fp32, or NULL
 * (then no workspace is used).
 * workspace: device, 256-byte aligned, >= qbmoe_add_rmsnorm_workspace_bytes(T, H)
 * bytes.  Sums are fp32 in a fixed order: bit-reproducible.  Rows whose squares, or products with g, pass fp32's
 * range or come near its least numbers are scaled by a power of two first; dn gamma itself is an fp32 number.
 *
 * 0 <= T <= QBMOE_MAX_ROWS, 1 <= H <= QBMOE_MAX_NORM, eps >= 0 and finite, row strides (ld*,
 * in elements) >= H.  Pointers are aligned to their element type only: rows whose bases and strides are
 * multiples of 16 bytes (and H of 8) are read as vectors.  codes are 8-byte aligned.
 */
int moe_add_rmsnorm(int T, int H, int x_type, const void* x, long long ldx, int res_type, const void* residual,
                    long long ldr, const float* gamma, float eps, void* total, long long ldt, void* y, long long ldy,
                    uint8_t* codes, uint8_t* scales, qbmoe_stream_t stream);
size_t qbmoe_add_rmsnorm_workspace_bytes(int T, int H);
int moe_add_rmsnorm_backward(int T, int H, int dn_type, const void* dn, long long lddn, int total_type,
                             const void* total, long long ldt, const float* gamma, float eps, const void* dtotal,
                             long long lddt, void* dx, long long lddx, float* dgamma, void* workspace,
                             size_t workspace_bytes, qbmoe_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * MXFP4 weights with few rows, and the routed experts of a few tokens.
 *
 * moe_mxfp4_matvec: y[r][f] = sum_k x[r][k] w[e(r)][f][k] with rows grouped as
 *   for moe_mxfp4_matmul (offsets [E + 1] or NULL; rows that no expert owns are not
 *   written), but x at its own precision: QBMOE_BF16 [R, K], row stride ldx, or
 *   QBMOE_MXFP8 (x the codes, x_scales the scales, ldx = K).  y [R, N] of y_type
 *   (QBMOE_BF16 or QBMOE_F32), row stride ldy.  Each expert's weights are read once per 8 of
 *   its rows, in pieces (below) once per 2, 8, 16 or 24, as many as R / E asks for: meant for few rows
 *   an expert.
 *   workspace: device, 256-byte aligned, >= qbmoe_mxfp4_matvec_workspace_bytes(R, N, K)
 *   bytes (0, and NULL allowed, for few rows and small weights up to K = 8192; it does not know E and
 *   holds what the largest would need).
 *
 * moe_mxfp4_experts: for T tokens with the experts idx [T, k] (an entry outside
 *   [0, E) stands for no route) and weights w [T, k] of moe_route_qb,
 *     a[t][i] = SiTU-GLU(x[t] w_gate[e]^T, x[t] w_up[e]^T),  e = idx[t][i]
 *     z[t]    = sum_i w[t][i] a[t][i] w_out[e]^T
 *     y[t]    = round(z) (gamma NULL), or round((z r) gamma), r = 1 / sqrt(mean z^2 + rms_eps)
 *   with SiTU-GLU of moe_latent_forward; beta1 and beta2 positive, beta1 beta2 at most 2^127,
 *   rms_eps finite and not negative; mean z^2 is an fp32 number.  x [T, L] as above, w_gate and w_up MXFP4
 *   [E, M, L], w_out [E, L, M], y [T, L] QBMOE_BF16 (row stride ldy), gamma [L] fp32.
 *   T k at most QBMOE_MAX_ROUTES.  workspace: device, 256-byte aligned, >=
 *   qbmoe_mxfp4_experts_workspace_bytes(T, k, L, M) bytes.
 *
 * Both take weights and MXFP8 rows as they are.  Small calls, and depths that are not multiples of 256 or
 * over 8192, take each block of 32 of a bf16 row as fp16 times a power of two: exact for elements
 * down to 2^-32 of the block's largest and within 2^-40 of it below; the SiTU-GLU's fp32 result as two such terms
 * (within 2^-22 of the value, or 2^-40 of the block's largest).  All others take bf16 rows, and the SiTU-GLU's
 * result, as sums of eight MXFP4 rows:
 * within 2^-22 of a block's largest (bf16 elements down to 2^-14 of it are exact); rows with
 * infinities or blocks of magnitudes below 2^-100 are multiplied as they are, slowly, and
 * what is below 2^-121 in the SiTU-GLU's result is dropped.  Sums are fp32 in a
 * fixed order: bit-reproducible (in pieces the tensor cores cut partial sums off where fp32 addition would
 * round).  So are a block's products before the weights' scale: where they pass fp32's range the result is infinite.  A row's result does not depend on other rows' elements.
 * 0 <= R <= QBMOE_MAX_ROWS, 1 <= E <= QBMOE_MAX_EXPERTS, 1 <= k <= QBMOE_MAX_TOPK, N a
 * multiple of 8, K, L and M multiples of 32 and at most QBMOE_MATVEC_MAX_K, E N below 2^31.  Pointers
 * 16-byte aligned (idx, w and gamma: 4), ldx a multiple of 8 elements; y aligned to its type.
 * A bounded wait that expires is reported by qbmoe_status(NULL, stream).
 */
#define QBMOE_MAX_NORM 16384
#define QBMOE_MAX_ROUTES 4096
#define QBMOE_MATVEC_MAX_K 65536
size_t qbmoe_mxfp4_matvec_workspace_bytes(int R, int N, int K);
int moe_mxfp4_matvec(int R, int E, int N, int K, int x_type, const void* x, long long ldx, const uint8_t* x_scales,
                     const uint8_t* w_codes, const uint8_t* w_scales, const int32_t* offsets, int y_type, void* y,
                     long long ldy, void* workspace, size_t workspace_bytes, qbmoe_stream_t stream);
size_t qbmoe_mxfp4_experts_workspace_bytes(int T, int k, int L, int M);
int moe_mxfp4_experts(int T, int k, int E, int L, int M, int x_type, const void* x, long long ldx,
                      const uint8_t* x_scales, const int32_t* idx, const float* w, const uint8_t* gate_codes,
                      const uint8_t* gate_scales, const uint8_t* up_codes, const uint8_t* up_scales,
                      const uint8_t* out_codes, const uint8_t* out_scales, float beta1, float beta2,
                      const float* gamma, float rms_eps, void* y, long long ldy, void* workspace,
                      size_t workspace_bytes, qbmoe_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Layer context.
 */
typedef struct {
    int d;              /* model width */
    int latent;         /* latent width ([K3-width] 延伸解读: 7168 -> 3584) */
    int n_experts;      /* routed experts */
    int top_k;          /* experts per token */
    int expert_inter;   /* routed expert GLU intermediate */
    int shared_inter;   /* merged shared-expert intermediate; 0 = no shared expert */
    float situ_beta1;   /* gate softcap, 4 on the pages */
    float situ_beta2;   /* up softcap, 25 on the pages */
    float rms_eps;      /* RMSNorm epsilon */
    int act_dtype;      /* QBMOE_F32 | QBMOE_BF16: activations and dense weights */
    int expert_wfmt;    /* QBMOE_W_F32 | QBMOE_W_BF16 | QBMOE_W_MXFP4 */
    int qb_sweeps;      /* 0 = frozen bias (inference); 1 = one QB step */
    int qb_mode;        /* QBMOE_QB_JACOBI (default) | QBMOE_QB_GAUSS_SEIDEL */
} qbmoe_config;

/*
 * Weights: device pointers in canonical K-major layouts ("[rows, K]", K
 * contiguous), typed by act_dtype unless stated.  The caller owns them and
 * must keep them alive and unchanged while the context uses them (the
 * context keeps pointers, not copies).
 *   w_router [n, d]; router_offset [n] fp32 or NULL (per-expert logit offset)
 *   w_down [latent, d]
 *   w_gate, w_up [n, m, latent]; w_out [n, latent, m]    (expert_wfmt)
 *     MXFP4: values packed two per byte (element 2i in the low nibble) as
 *     [rows, K/2] u8 with 32-byte aligned bases, scales E8M0 [rows, K/32]
 *     u8 in s_gate/s_up/s_out (tensor-core path: K a multiple of 512).
 *   rms_gamma [latent] fp32
 *   w_proj_up [d, latent]
 *   w_shared_gate, w_shared_up [m_s, d]; w_shared_out [d, m_s]  (m_s > 0)
 */
typedef struct {
    const void* w_router;
    const float* router_offset;
    const void* w_down;
    const void* w_gate;
    const void* w_up;
    const void* w_out;
    const uint8_t* s_gate;
    const uint8_t* s_up;
    const uint8_t* s_out;
    const float* rms_gamma;
    const void* w_proj_up;
    const void* w_shared_gate;
    const void* w_shared_up;
    const void* w_shared_out;
} qbmoe_weights;

typedef struct qbmoe_ctx qbmoe_ctx;

/* Validate cfg, allocate the context's device workspace for up to max_tokens
 * tokens on the current device (synchronous).  *out = NULL on failure. */
int qbmoe_create(qbmoe_ctx** out, const qbmoe_config* cfg, int max_tokens);
/* Bytes of device workspace qbmoe_create allocates for these sizes. */
size_t qbmoe_layer_workspace_bytes(const qbmoe_config* cfg, int max_tokens);
/* Record the weight pointers (host call, no device work, no copies). */
int qbmoe_set_weights(qbmoe_ctx* ctx, const qbmoe_weights* w);
/* Copy the weights into device memory the context owns, then use the
 * copies (as qbmoe_set_weights on them).  w holds device pointers in the
 * layouts above; the caller may free or change its tensors once the call
 * returns.  Synchronous: enqueues the copies and a check of every MXFP4
 * scale byte on `stream`, then waits for them.  A scale byte of 0xFF (E8M0
 * NaN, not a weight scale) gives QBMOE_EINVAL and leaves the context's
 * weights as they were.  Allocates one buffer (cudaMalloc; QBMOE_ENOMEM on
 * failure); a later call replaces it, qbmoe_destroy frees it.  Nothing else
 * in the forward path allocates. */
int qbmoe_pack_weights(qbmoe_ctx* ctx, const qbmoe_weights* w, qbmoe_stream_t stream);
/* Free the context's workspace (synchronous). NULL is a no-op. */
int qbmoe_destroy(qbmoe_ctx* ctx);

/*
 * moe_latent_forward — one Stable LatentMoE layer forward for T tokens.
 *
 *   scores = sigmoid(x W_r^T + o) (or of logits_in when given)   [K3-width] Q&A routing
 *   b, idx, w, loads as moe_route_qb
 *   h   = round(x W_down^T)                                       [K3-width] 延伸解读 latent
 *   act = round(SiTU-GLU(h W_g[e]^T, h W_u[e]^T)) per route       [K3-width] Q&A SiTU-GLU
 *         SiTU-GLU(g, u) = a*sigmoid(a)*b, a = b1*tanh(g/b1), b = b2*tanh(u/b2)
 *   e   = round(act W_o[e]^T)
 *   z   = round(RMSNorm(sum_i w_i e_i) * gamma)                   [K3-width] Q&A RMSNorm
 *   out = round(z W_proj_up^T + act_s W_shared_out^T),
 *         act_s = round(SiTU-GLU(x W_shared_gate^T, x W_shared_up^T))   Q&A shared expert
 * ("round" = to act_dtype; accumulation is fp32.  With bf16 activations the
 * tensor-core SiTU epilogues use the hardware tanh approximation, relative
 * error about 2^-11, below the bf16 rounding.  MXFP4 experts run on the
 * block-scaled MMA: each block of 32 bf16 activations along K gets an E8M0
 * scale 2^e, e = floor(log2 max|a|) - 7, and each scaled value c = a 2^-e
 * (|c| < 256) enters as e4m3(c) + e4m3(16 (c - e4m3(c))) / 16, which is
 * exact for 2^-6 <= |c| < 256; nothing saturates.)
 *
 * x [T, d] act_dtype device; out [T, d] act_dtype device.
 * logits_in: NULL, or [T, n] fp32 device router logits used instead of the
 *   router GEMM (x W_r^T + o is then not computed).
 * bias_in [n] fp32 device or NULL (zeros); bias_out [n] fp32 device (may
 *   alias bias_in) or NULL.
 * scores_opt [T, n] fp32, idx_opt [T, k] int32, w_opt [T, k] fp32,
 *   loads_opt [n] int32: device outputs, each NULL if not wanted.
 * 1 <= T <= max_tokens.  No allocation, no host synchronisation.
 * With qb_mode = QBMOE_QB_GAUSS_SEIDEL the qb_sweeps sweeps are cyclic, as
 * moe_route_qb_gs (about 2n launches per sweep).
 */
int moe_latent_forward(qbmoe_ctx* ctx, int T, const void* x, const float* logits_in,
                       const float* bias_in, float* bias_out, void* out,
                       float* scores_opt, int32_t* idx_opt, float* w_opt, int32_t* loads_opt,
                       qbmoe_stream_t stream);

/*
 * Synchronise `stream`, then return and clear the context's device status
 * word: QBMOE_OK, QBMOE_ETIMEOUT (a bounded wait expired; the kernel
 * returned early and its outputs are undefined) or QBMOE_EDEVICE.
 * ctx may be NULL: QBMOE_ETIMEOUT if a bounded wait of any call that takes no
 * context (moe_mxfp4_*) has expired on the current device since the calling
 * host thread last asked, in whichever thread or stream (a thread that never
 * asked: since the library was loaded).
 */
int qbmoe_status(qbmoe_ctx* ctx, qbmoe_stream_t stream);

/*
 * Stage timing.  qbmoe_set_timing(ctx, slots) (synchronous) keeps CUDA events
 * around each stage of the next `slots` forwards (a ring; 0 = off, at most
 * 4096) on the forward's stream, without synchronising.  qbmoe_stage_times
 * (synchronous) writes each stage's mean milliseconds over the recorded
 * forwards still in the ring into ms[0..max-1] and the stages' names (static
 * strings) into names (may be NULL); returns the number of stages, 0 if none.
 */
int qbmoe_set_timing(qbmoe_ctx* ctx, int slots);
int qbmoe_stage_times(qbmoe_ctx* ctx, float* ms, const char** names, int max);

/* Number of kernels the last moe_latent_forward / moe_route_qb call launched. */
int qbmoe_last_launch_count(qbmoe_ctx* ctx);
int qbmoe_route_last_launch_count(void);

/* Test hook: cap on bounded device waits, in polls of at most 20 us each
 * (<= 0 restores the default of 2^17).  Applies to launches made after the
 * call.  ctx NULL: the moe_mxfp4_* calls of the calling host thread. */
int qbmoe_set_wait_limit(qbmoe_ctx* ctx, long long iterations);

/* Test hook: while enabled, the tensor-core GEMM kernels withhold their first
 * accumulator hand-off, so the epilogue's bounded wait expires and the next
 * qbmoe_status reports QBMOE_ETIMEOUT (outputs undefined).  The kernels then
 * drain their own copies and MMAs, free TMEM and return; the context stays
 * usable.  No effect when the layer runs on CUDA cores.  ctx NULL: the
 * moe_mxfp4_* products that the calling host thread makes. */
int qbmoe_debug_stall(qbmoe_ctx* ctx, int enable);

/* 1 when the context's bf16 GEMMs run on the tcgen05 tensor-core kernels, 0
 * when they run on the CUDA-core kernels (fp32 layers, shapes the tensor-core
 * tiling does not cover, or QBMOE_DISABLE_TC=1 in the environment at
 * qbmoe_create). */
int qbmoe_uses_tensor_cores(qbmoe_ctx* ctx);

/*
 * Tensor-core rate probe (synchronous; a measurement hook, not part of the
 * layer).  Runs one CTA per SM that issues 4 * iters back-to-back MMAs of
 * the given kind on fixed shared-memory tiles (M = 128, N = 256; no TMA, no
 * epilogue) between two CUDA events on the legacy default stream.  Kinds:
 * QBMOE_PROBE_BF16 (kind::f16, bf16 x bf16, K = 16 per MMA) and
 * QBMOE_PROBE_MXF4F8 (kind::mxf8f6f4 block-scaled, E2M1 x E4M3 with E8M0
 * scales, K = 32 per MMA: the MXFP4 expert GEMMs' instruction).  Writes the
 * elapsed milliseconds and the flops issued (2 * M * N * K per MMA).
 * Allocates a 4-byte status word (cudaMalloc) for its bounded wait.
 */
enum { QBMOE_PROBE_BF16 = 0, QBMOE_PROBE_MXF4F8 = 1 };
int qbmoe_mma_probe(int kind, int iters, float* ms_out, double* flops_out);

const char* qbmoe_strerror(int code);

#ifdef __cplusplus
}
#endif
#endif /* QBMOE_H */
