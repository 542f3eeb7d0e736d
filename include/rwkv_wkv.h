/*
 * rwkv_wkv.h -- C ABI of libwkv.so: the WKV time-mixing recurrences of RWKV-4 and
 * Eagle/Finch (RWKV-5/6) on NVIDIA B200 (sm_100a).
 *
 * Sources (page title, section):
 *  [R4]   "RWKV: Reinventing RNNs for the Transformer Era" (Chinese translation):
 *         section "类 Transformer 的并行化" (time-parallel mode: the WKV update is a
 *         serial scan of cost O(BTd)); section "梯度稳定性和层堆叠" (single-step
 *         time-dependent softmax); section "利用时间结构进行时序数据处理" (time decay
 *         e^{-w} and bonus e^{u} of eq. 14); section "类 RNN 的序列解码" (RNN-mode
 *         decoding with constant memory per token).
 *  [E412] "RWKV-5/6 (Eagle and Finch)", section 4.1.2 (Eagle time mixing): matrix-valued
 *         state s = sum of k^T v, decayed per key channel by w, gain u on the current
 *         token, receptance as a query; w = exp(-exp(omega)) in (0,1).  Section 4 fixes
 *         row vectors with matrices acting on the right.
 *  [F422] same page, section 4.2.2 (Finch time mixing): w_t varies per token and channel.
 *
 * Conventions shared by every entry point
 *  - All tensor pointers are DEVICE pointers owned by the caller, dense and row-major
 *    with the channel index innermost.  The library never allocates, frees or retains
 *    them; it reads inputs and writes outputs asynchronously on the calling thread's
 *    stream (rwkv_set_stream) and returns before the GPU has finished.
 *  - bf16 tensors are passed as uint16_t bit patterns (IEEE bfloat16, round-to-nearest-
 *    even on output).  Accumulation is fp32 throughout.
 *  - Every tensor pointer must be 16-byte aligned (RWKV_ERR_ALIGN otherwise).
 *  - Sizes are int64_t and must be >= 0 (RWKV_ERR_SHAPE otherwise).  A call with no
 *    output element to produce returns RWKV_OK without launching; for T == 0 the final
 *    state is still written (a copy of s0, or the empty state).
 *  - A pointer may be NULL only where stated, or when the tensor it names is empty.
 *  - Outputs must not overlap any input (RWKV_ERR_ALIAS), except that a state output
 *    may be the very same pointer as the state input (in-place state update).
 *  - Return value: RWKV_OK (0) or a negative rwkv_status.  Argument errors are found
 *    on the host before any CUDA call.  RWKV_ERR_CUDA means a launch or CUDA runtime
 *    call failed; rwkv_last_error() has the text.  Faults inside a kernel that the
 *    kernel itself detects (e.g. a bounded wait that ran out) are reported through the
 *    device status word, read with rwkv_get_device_status().
 *  - The library keeps no device memory of its own beyond its status word and the fixed
 *    scratch array of rwkv_wkv6_forward_bf16_noalloc (statically allocated __device__
 *    variables).  The only per-call allocation is the stream-ordered scratch of a split
 *    chunked WKV-6 call (see rwkv_set_wkv6_segments); the backward pass takes its
 *    workspace from the caller.
 */
#ifndef RWKV_WKV_H
#define RWKV_WKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RWKV_ABI_VERSION 1

typedef enum rwkv_status {
    RWKV_OK = 0,
    RWKV_ERR_NULL = -1,        /* a required pointer is NULL                          */
    RWKV_ERR_SHAPE = -2,       /* a negative size, or a size product overflows        */
    RWKV_ERR_UNSUPPORTED = -3, /* e.g. WKV-6 head size N != 64                        */
    RWKV_ERR_ALIAS = -4,       /* an output overlaps an input                         */
    RWKV_ERR_CUDA = -5,        /* a CUDA runtime call or kernel launch failed         */
    RWKV_ERR_TIMEOUT = -6,     /* a bounded device-side wait ran out (device status)  */
    RWKV_ERR_ALIGN = -7,       /* a tensor pointer is not 16-byte aligned             */
    RWKV_ERR_ARG = -8,         /* another invalid argument (e.g. unknown option)      */
    RWKV_ERR_BOUNDS = -9       /* debug build only: a kernel's index check failed and
                                  the access was skipped (device status)              */
} rwkv_status;

/* ------------------------------------------------------------------ RWKV-4 WKV [R4]
 * Per batch row b and channel c, with keys k_t, values v_t:
 *   y_t = ( sum_{i<t} e^{-(t-1-i) w_c + k_i} v_i + e^{u_c + k_t} v_t )
 *       / ( sum_{i<t} e^{-(t-1-i) w_c + k_i}     + e^{u_c + k_t}     )
 * evaluated in the running-maximum (time-dependent softmax) form, so k may be large.
 *   w, u : [C] fp32.  w is the positive decay RATE (per-step factor e^{-w}); the
 *          library does not exponentiate a learned parameter for you.
 *   k, v : [B, T, C];  y : [B, T, C] (same dtype as k).
 */
int rwkv_wkv4_forward(int64_t B, int64_t T, int64_t C,
                      const float *w, const float *u,
                      const float *k, const float *v, float *y);
int rwkv_wkv4_forward_bf16(int64_t B, int64_t T, int64_t C,
                           const float *w, const float *u,
                           const uint16_t *k, const uint16_t *v, uint16_t *y);

/* RWKV-4 WKV with state carry, so a sequence can be split across calls exactly
 * ([R4] RNN-mode decoding).  State layout s0/sT: [B, 3, C] fp32 = (a, b, p) per
 * channel, meaning numerator = a e^p and denominator = b e^p of the decayed past sums
 * after the last token processed.  An empty state has a = b = 0 (p is then ignored;
 * the library writes p = -1e30 for it).  s0 NULL = empty state; sT NULL = not written;
 * sT may equal s0.  The (a, b, p) triple is not unique: compare states through
 * a e^{p-P}, b e^{p-P} at a common P. */
int rwkv_wkv4_forward_state(int64_t B, int64_t T, int64_t C,
                            const float *w, const float *u,
                            const float *k, const float *v,
                            const float *s0, float *y, float *sT);
int rwkv_wkv4_forward_state_bf16(int64_t B, int64_t T, int64_t C,
                                 const float *w, const float *u,
                                 const uint16_t *k, const uint16_t *v,
                                 const float *s0, uint16_t *y, float *sT);

/* ------------------------------------------------------- Eagle/Finch WKV-6 [E412][F422]
 * Per batch row b and head h, state S (N x N, row i = key channel, column j = value
 * channel), for t = 0..T-1:
 *   y_t[j] = sum_i r_t[i] ( S[i][j] + u[i] k_t[i] v_t[j] )
 *   S[i][j] <- w_t[i] S[i][j] + k_t[i] v_t[j]
 * with S = s0 before the first token and sT = S after the last.
 *   r, k, v, w, y : [B, T, H, N]; w_t in (0, 1] (Eagle: constant over t; Finch: per
 *                   token).  w outside (0, 1] is outside the contract: results are then
 *                   unspecified but the call never faults.
 *   u             : [H, N] fp32.
 *   s0, sT        : [B, H, N, N] fp32.  s0 NULL = zero state; sT NULL = not written;
 *                   sT may equal s0 (in-place).
 *   N must be 64 (RWKV_ERR_UNSUPPORTED otherwise).
 * fp32 inputs run a serial fp32 kernel (SIMT).  bf16 inputs with T > 1 run the chunked
 * tensor-core kernel (64-token chunks, bf16 operands, fp32 accumulation, state in fp32);
 * T == 1 runs the bandwidth-bound decode kernel.
 */
int rwkv_wkv6_forward(int64_t B, int64_t T, int64_t H, int64_t N,
                      const float *r, const float *k, const float *v, const float *w,
                      const float *u, const float *s0, float *y, float *sT);
int rwkv_wkv6_forward_bf16(int64_t B, int64_t T, int64_t H, int64_t N,
                           const uint16_t *r, const uint16_t *k, const uint16_t *v,
                           const uint16_t *w, const float *u, const float *s0,
                           uint16_t *y, float *sT);

/* WKV-6 with the time-mixing output stage fused into the epilogue ([E412]: LayerNorm on
 * each head, i.e. GroupNorm over the H heads, then the SiLU attention gate):
 *   o = the rwkv_wkv6_forward_bf16 output (fp32 before rounding),
 *   y[b,t,h,:] = SiLU(g[b,t,h,:]) * ( ln_w[h,:] * (o - mean) / sqrt(var + eps) + ln_b[h,:] )
 * with mean and var (mean of squared deviations) over the N channels of o[b,t,h,:] and
 * SiLU(x) = x / (1 + e^-x).  y is written once, in bf16; the state is as in
 * rwkv_wkv6_forward_bf16.
 *   g             : [B, T, H, N] bf16, the gate before its activation; must not overlap y.
 *   ln_w, ln_b    : [H, N] fp32, the per-channel scale and shift (not NULL).
 *   eps           : >= 0 (RWKV_ERR_ARG otherwise).
 * T > 1 runs the chunked kernel, T == 1 the decode kernel, each with the fused epilogue
 * (the rwkv_set_wkv6_algo choice does not apply).  Other arguments, layouts, aliasing
 * rules and errors are those of rwkv_wkv6_forward_bf16. */
int rwkv_wkv6_forward_gated_bf16(int64_t B, int64_t T, int64_t H, int64_t N,
                                 const uint16_t *r, const uint16_t *k, const uint16_t *v,
                                 const uint16_t *w, const float *u, const float *s0,
                                 const uint16_t *g, const float *ln_w, const float *ln_b, float eps,
                                 uint16_t *y, float *sT);

/* WKV-6 fed the decay LOGIT instead of the decay ([E412]: w = exp(-exp(omega)) with omega
 * the trainable per-head parameter; [F422]: omega_t per token, the learned omega plus the
 * data-dependent LoRA offset of the Finch token shift, section 4.2.1).  The kernels form
 *   w_t[i] = exp(-exp(omega_t[i]))
 * in fp32 as they load each tile and then run the recurrence of rwkv_wkv6_forward_bf16.
 * Passing omega_t saves the caller a separate elementwise pass over [B, T, H, N], and a decay
 * close to 1 keeps its distance from 1: a bf16 w cannot hold one (the largest bf16 value
 * below 1 is 1 - 2^-8), so slowly decaying channels of a bf16 w round to w = 1 or to
 * 1 - 2^-8.  Any omega, +-inf included, gives w in [0, 1]; NaN is outside the contract.
 *   omega         : [B, T, H, N] bf16 (in place of w).
 *   g, ln_w, ln_b : all NULL = plain output (as rwkv_wkv6_forward_bf16);  all non-NULL =
 *                   the fused head LayerNorm + SiLU gate of rwkv_wkv6_forward_gated_bf16,
 *                   with eps as there.  Some but not all NULL: RWKV_ERR_NULL.  eps is
 *                   ignored without the gate.
 * Kernels, the rwkv_set_wkv6_algo choice (plain output only), layouts, aliasing rules and
 * errors are those of rwkv_wkv6_forward_bf16 / rwkv_wkv6_forward_gated_bf16.  The chunked
 * kernel forms w_t with the hardware's approximate base-2 exponential (relative error of
 * order 1e-7 on w_t); the serial and decode kernels with the accurate one. */
int rwkv_wkv6_forward_omega_bf16(int64_t B, int64_t T, int64_t H, int64_t N,
                                 const uint16_t *r, const uint16_t *k, const uint16_t *v,
                                 const uint16_t *omega, const float *u, const float *s0,
                                 const uint16_t *g, const float *ln_w, const float *ln_b, float eps,
                                 uint16_t *y, float *sT);

/* WKV-6 backward pass, for training ([E412], [F422]; the gradients of the recurrence of
 * rwkv_wkv6_forward by the chain rule, walked backwards in time).  Given the gradients of a
 * loss L with respect to the forward's outputs,
 *   dy  = dL/dy  [B, T, H, N] (dtype of r),   dsT = dL/dsT [B, H, N, N] fp32 (NULL = 0),
 * it writes, all fp32:
 *   dr, dk, dv, dw : [B, T, H, N]   dL/dr, dL/dk, dL/dv, dL/dw per token and channel
 *                    (rwkv_wkv6_backward_omega_bf16: domega = dL/domega_t in place of dw);
 *   du             : [H, N]         dL/du, summed over the batch rows in a fixed order
 *                                   (deterministic);
 *   ds0            : [B, H, N, N]   dL/ds0, or NULL = not written.  ds0 may be the very
 *                                   same array as dsT (in place).
 * With L_t = dL/d(state after token t), L_{T-1} = dsT and S = the state before token t:
 *   dr_t[i] = sum_j dy_t[j] (S[i][j] + u[i] k_t[i] v_t[j])
 *   dk_t[i] = sum_j L_t[i][j] v_t[j] + u[i] r_t[i] (dy_t . v_t)
 *   dv_t[j] = sum_i L_t[i][j] k_t[i] + (sum_i r_t[i] u[i] k_t[i]) dy_t[j]
 *   dw_t[i] = sum_j L_t[i][j] S[i][j]           domega_t[i] = -dw_t[i] exp(omega_t[i]) w_t[i]
 *   du[i]   = sum_{b,t} r_t[i] k_t[i] (dy_t . v_t)
 *   L_{t-1} = diag(w_t) L_t + r_t^T dy_t,       ds0 = L_{-1}.
 * Inputs r, k, v, w (or omega), u, s0 are those of the forward call; the forward states
 * are recomputed, not read.
 *   workspace : device scratch owned by the caller, 16-byte aligned, of at least the size
 *               rwkv_wkv6_backward_workspace_bytes reports (about B*H*ceil(T/8)*N*N*4 bytes:
 *               room for an fp32 checkpoint of the state every 8 tokens, which the exact
 *               walks below use; the chunked path needs about an eighth of it); it must not
 *               overlap any tensor.  A smaller workspace_bytes is refused with RWKV_ERR_ARG
 *               before any launch.  Its contents need no initialisation and are undefined
 *               after the call.
 * Two paths (rwkv_set_wkv6_algo on the calling thread chooses):
 *   - bf16 inputs (default, and RWKV_WKV6_AUTO / RWKV_WKV6_CHUNKED): the chunked tensor-core
 *     path in 64-token chunks -- a pass over the chunks for the state entering each chunk
 *     (kept in bf16), a reverse pass for the state gradient leaving each chunk, and one
 *     kernel over all (b, h, chunk) at once for the gradients, with bf16 MMA operands and
 *     fp32 accumulation (results within the bf16 tolerance of the exact gradient).  A (b, h)
 *     sequence with a channel whose 64-token decay product falls below 2^-100, or (w input)
 *     with a w below 2^-5, is served by the exact walks instead, inside the same call.
 *   - fp32 inputs, or RWKV_WKV6_SERIAL: the exact walks on CUDA cores in fp32 (a forward
 *     pass for dr, du and the checkpoints; a backward pass over state rows for dk, dw; one
 *     over state columns for dv, ds0).
 * du is summed over the batch rows (and chunks) in a fixed order: results are deterministic.
 * N must be 64.  T = 0 writes du = 0 and ds0 = dsT.  Aliasing: no output may overlap an
 * input, the workspace or another output (except ds0 == dsT).  Other rules and errors as
 * rwkv_wkv6_forward. */
int rwkv_wkv6_backward_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t N, size_t *bytes);
int rwkv_wkv6_backward(int64_t B, int64_t T, int64_t H, int64_t N,
                       const float *r, const float *k, const float *v, const float *w,
                       const float *u, const float *s0, const float *dy, const float *dsT,
                       float *dr, float *dk, float *dv, float *dw, float *du, float *ds0,
                       void *workspace, size_t workspace_bytes);
int rwkv_wkv6_backward_bf16(int64_t B, int64_t T, int64_t H, int64_t N,
                            const uint16_t *r, const uint16_t *k, const uint16_t *v,
                            const uint16_t *w, const float *u, const float *s0,
                            const uint16_t *dy, const float *dsT,
                            float *dr, float *dk, float *dv, float *dw, float *du, float *ds0,
                            void *workspace, size_t workspace_bytes);
int rwkv_wkv6_backward_omega_bf16(int64_t B, int64_t T, int64_t H, int64_t N,
                                  const uint16_t *r, const uint16_t *k, const uint16_t *v,
                                  const uint16_t *omega, const float *u, const float *s0,
                                  const uint16_t *dy, const float *dsT,
                                  float *dr, float *dk, float *dv, float *domega, float *du,
                                  float *ds0, void *workspace, size_t workspace_bytes);

/* ------------------------------------------------------------------ gated delta rule
 * The recurrence whose state is corrected towards each new value instead of only decayed:
 * per sequence and value head h, state S (N x N, row i = key channel, column j = value
 * channel, as in WKV-6), for each token t:
 *   S'  = exp(g_t) S                       decay, one factor per token and head
 *   u_t = beta_t (v_t - k_t S')            what k_t does not recall yet of v_t
 *   S   = S' + k_t^T u_t
 *   o_t = scale q_t S                      (reads the state after the token's update)
 * with S = s0 before the first token and sT = S after the last.
 *   q, k    : [B, T, Hk, N];   v, o : [B, T, H, N].  Hk divides H; value head h uses key
 *             head h / (H / Hk).  Queries and keys are used as given (the caller
 *             normalises them).
 *   g, beta : [B, T, H], in the type of q: the log of the decay (<= 0 for a decay; -inf
 *             forgets the state) and the gate of the update.
 *   scale   : finite (RWKV_ERR_ARG otherwise).
 *   offsets : NULL: the B rows are the sequences.  Otherwise int32 [nseq + 1] on the device,
 *             and B must be 1: sequence i is the tokens offsets[i] .. offsets[i+1] - 1 of
 *             the T packed ones (ascending; a sequence may be empty).  Tokens outside every
 *             sequence are neither read nor written.  Values outside 0 .. T are clamped.
 *             nseq is ignored without offsets.
 *   s0, sT  : fp32, NULL = zero state / not written; sT may equal s0 (in place).  Without
 *             slots, [nseq, H, N, N].  With slots, a pool [nslots, H, N, N] where sequence i
 *             uses state slots[i] (int32 [nseq] on the device); the other slots are neither
 *             read nor written.  A negative slot means no state: the sequence starts from
 *             zero and its last state is dropped (a padding row of a decode batch).  A slot
 *             past the pool does the same and records RWKV_ERR_ARG in the device status
 *             word.  A slot named by two sequences of one call ends with the state of one
 *             of them, or, in place, of either started from any mix of the two: name each
 *             slot once (rwkv_state_copy forks states).  nslots is ignored without slots.
 *   workspace : device scratch owned by the caller, 16-byte aligned, of at least the bytes
 *             that rwkv_delta_forward_workspace_bytes reports for the same sizes (packed:
 *             offsets given; bf16: the entry point's type); fewer are refused with
 *             RWKV_ERR_ARG.  Zero bytes (workspace may be NULL) for fp32 and for short
 *             sequences.  No initialisation needed, undefined afterwards; calls whose work
 *             overlaps need a workspace each.
 *   N must be 64.  Index arrays are 4-byte aligned; other rules and errors as above.
 *   Inputs of the tokens that sequences hold are finite (g may be -inf).  One that is not may
 *   reach the outputs of up to 63 tokens before it too: give padding tokens zeros.
 * Accumulation is fp32 and the state is held in fp32 throughout.  bf16 sequences of 24 tokens
 * or more (packed: on average) run in 64-token chunks on the tensor cores: there the output
 * is formed from bf16 operands, and every operand of the state from two bf16 terms (2^-16 of
 * its value).  Others run token by token in fp32, 0.23 us a token; fp32 copies of bf16 inputs do
 * so whatever their length.  The choice is made for the whole call, from T / nseq: the bits of a
 * packed sequence can depend on its neighbours, and one long sequence among many short ones is
 * walked token by token.  Give it a call of its own over its part of the arrays (2048 tokens
 * beside 127 single ones, 16 heads, bf16: 631 us in one call, 73 and 15 us in two).
 */
int rwkv_delta_forward_workspace_bytes(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N,
                                       int64_t nseq, int packed, int bf16, size_t *bytes);
int rwkv_delta_forward(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N,
                       const float *q, const float *k, const float *v, const float *g,
                       const float *beta, float scale, int64_t nseq, const int32_t *offsets,
                       int64_t nslots, const int32_t *slots, const float *s0, float *o,
                       float *sT, void *workspace, size_t workspace_bytes);
int rwkv_delta_forward_bf16(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N,
                            const uint16_t *q, const uint16_t *k, const uint16_t *v,
                            const uint16_t *g, const uint16_t *beta, float scale, int64_t nseq,
                            const int32_t *offsets, int64_t nslots, const int32_t *slots,
                            const float *s0, uint16_t *o, float *sT, void *workspace,
                            size_t workspace_bytes);

/* Backward pass of the gated delta rule.  Given dout = dL/do ([B, T, H, N], type of q) and
 * dsT = dL/dsT ([nseq, H, N, N] fp32, NULL = 0) it writes, with D the gradient of the state
 * after token t, r_t = v_t - k_t S' and S the state after token t:
 *   D += scale q_t^T do_t;   du = k_t D
 *   dq_t = scale S do_t^T    dv_t = beta_t du         dbeta_t = du . r_t
 *   dk_t = D u_t^T - S' dv_t^T   (dq and dk summed over the value heads of a key head)
 *   D' = D - k_t^T dv_t      dg_t = sum_ij D' S'      D <- exp(g_t) D'
 *   ds0 = D before the first token.
 *   dq, dk : [B, T, Hk, N];  dv : [B, T, H, N];  dg, dbeta : [B, T, H], in the type of the
 *            inputs;  ds0 : [nseq, H, N, N] fp32, NULL = not written; may equal dsT.
 *   Gradients of tokens outside every sequence are not written.
 *   workspace : device scratch owned by the caller, 16-byte aligned, of at least the bytes
 *            that rwkv_delta_backward_workspace_bytes reports for the same sizes (packed:
 *            offsets given; bf16: the entry point's type); fewer are refused with
 *            RWKV_ERR_ARG.  No initialisation needed, undefined afterwards; calls whose work
 *            overlaps need a workspace each.  For each token and value head it holds 768 bytes
 *            (bf16 sequences of 9 tokens or more, packed: on average) or 4 KB (others, 4.3 GB at
 *            B8 T4096 H32; none for rows of up to 8 tokens), and 512 more where key heads are
 *            shared; a sequence's last chunk of 64 tokens, or segment of 8, counts whole.
 * Results are deterministic.  No output may overlap an input, the workspace or another
 * output (except ds0 == dsT).  Other rules as rwkv_delta_forward. */
int rwkv_delta_backward_workspace_bytes(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N,
                                        int64_t nseq, int packed, int bf16, size_t *bytes);
int rwkv_delta_backward(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N,
                        const float *q, const float *k, const float *v, const float *g,
                        const float *beta, float scale, int64_t nseq, const int32_t *offsets,
                        const float *s0, const float *dout, const float *dsT, float *dq,
                        float *dk, float *dv, float *dg, float *dbeta, float *ds0,
                        void *workspace, size_t workspace_bytes);
int rwkv_delta_backward_bf16(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N,
                             const uint16_t *q, const uint16_t *k, const uint16_t *v,
                             const uint16_t *g, const uint16_t *beta, float scale, int64_t nseq,
                             const int32_t *offsets, const float *s0, const uint16_t *dout,
                             const float *dsT, uint16_t *dq, uint16_t *dk, uint16_t *dv,
                             uint16_t *dg, uint16_t *dbeta, float *ds0, void *workspace,
                             size_t workspace_bytes);

/* ------------------------------------------------------------------ pools of states
 * A serving process keeps the recurrent states of its sequences in the slots of a pool,
 * [layers, nslots, slot_bytes], of any of the state layouts above (slot_bytes a multiple of
 * 16, RWKV_ERR_ALIGN otherwise).
 *
 * rwkv_state_copy: for the n pairs (n <= 4096, RWKV_ERR_SHAPE otherwise), in every layer,
 *   slot dst[i] <- slot src[i] as it was before the call
 * so that any set of pairs, swaps and shifts included, is one call.  One src in several
 * pairs forks a state; src[i] < 0 frees dst[i] (zeros it: the empty state of WKV-6 and the
 * delta rule); dst[i] < 0 leaves the pair out.  Where several pairs name one dst, the last
 * of them counts.  A pair with an index past the pool is left out and RWKV_ERR_ARG recorded
 * in the device status word.  src, dst: int32 [n] on the device.
 *
 * rwkv_state_compact: moves the live slots (live[i] != 0, one byte each) to the front of the
 * pool in their order, in every layer: new_index[i] = the number of live slots before slot
 * i, or -1 if it is not live, and *count = the number of live slots.  The slots from *count
 * on keep what they hold.  nslots <= 16384 (RWKV_ERR_SHAPE otherwise).  live, new_index
 * ([nslots] int32) and count (int32) are on the device.
 *
 * Both are asynchronous and allocate nothing.  The arrays must not overlap one another.  A copy
 * holds a piece of every source of the call at once: from a few dozen sources on the pieces are
 * small, and with thousands of pairs finding each pair's part takes longer than the bytes
 * (src/dst permutations over 12 layers: 256 states of 32 heads 1.7 ms, 1.9 TB/s; 4096 of one
 * head 23 ms). */
int rwkv_state_copy(int64_t layers, int64_t nslots, int64_t slot_bytes, void *pool, int64_t n,
                    const int32_t *src, const int32_t *dst);
int rwkv_state_compact(int64_t layers, int64_t nslots, int64_t slot_bytes, void *pool,
                       const uint8_t *live, int32_t *new_index, int32_t *count);

/* Kernel choice for WKV-6 on the calling thread: RWKV_WKV6_AUTO (default, as above),
 * RWKV_WKV6_SERIAL (always the serial kernel; the backward takes the exact fp32 walks),
 * RWKV_WKV6_CHUNKED (the chunked kernel for bf16 whatever T; ignored for fp32).  Returns
 * RWKV_OK or RWKV_ERR_ARG. */
#define RWKV_WKV6_AUTO 0
#define RWKV_WKV6_SERIAL 1
#define RWKV_WKV6_CHUNKED 2
int rwkv_set_wkv6_algo(int algo);
int rwkv_get_wkv6_algo(void);

/* Sequence split of the chunked WKV-6 kernel on the calling thread.  Each (b, h) sequence
 * is walked by one CTA; when there are fewer sequences than two per SM the library cuts
 * every sequence into G segments (of at least four 64-token chunks) that run side by
 * side: a first pass gives the end state (from zero) and decay product of P pieces of each
 * segment but the last (P = 1, 2, 4 ...: halves while the pieces keep at least four chunks
 * and the first pass fits on the GPU at once), and each segment then starts from its exact
 * incoming state.  The result equals the unsplit evaluation up to fp32 rounding order.  The
 * split needs B*H*(G-1)*P*(N*N+N)*4 bytes of scratch, plus B*H*N*N*4 bytes for a copy of s0
 * when the state is updated in place
 * (sT == s0: the copy is taken before any segment runs, so no segment can read an s0 that
 * the last segment has already overwritten).  The scratch is taken stream-ordered (on the
 * calling thread's stream, within the call) from a memory pool the library keeps per
 * device, which holds up to 64 MB between calls.
 *   segments = 0 (default): choose G;  1: never split;  n >= 2: split into at most n.
 * Returns RWKV_OK or RWKV_ERR_ARG. */
int rwkv_set_wkv6_segments(int segments);
int rwkv_get_wkv6_segments(void);

/* Allocation-free variant of rwkv_wkv6_forward_bf16 (the paper has no counterpart: it is
 * a service of this library).  Some callers may not allocate device memory at all -- a
 * serving process that has handed its whole HBM budget to its own pool, code that must
 * not touch the allocator while other work is in flight, or a runtime that forbids
 * allocation outside its own set-up phase.  For them this call runs the chunked kernel with
 * the same sequence split as the default entry point, but keeps the split's scratch in a
 * fixed array inside the library (RWKV_NOALLOC_SCRATCH_BYTES per GPU, held by every GPU
 * that loads the library until the process exits) and never allocates or frees memory.
 *   segments: 0 = choose the split as rwkv_wkv6_forward_bf16 does, capped to what the
 *             array holds; n >= 1 = split into at most n segments.  The first pass uses
 *             P pieces per segment as the default entry point does, fewer (down to 1) when
 *             their entries would not fit.  A split needing more than
 *             RWKV_NOALLOC_SCRATCH_BYTES (B*H*(G-1)*P*(N*N+N)*4 bytes for G segments,
 *             plus B*H*N*N*4 bytes for the copy of s0 when sT == s0) is rejected with
 *             RWKV_ERR_SHAPE before any launch; rwkv_last_error() says why.
 * Arguments, layouts and the result are otherwise those of rwkv_wkv6_forward_bf16 (always
 * the chunked kernel, whatever T).
 *   - The first call on each device looks up the array's device address (a CUDA runtime
 *     query, no allocation); make that first call before capturing a stream into a graph.
 *   - Every call shares the one array and it keeps what the last call left; the kernels
 *     write every scratch entry before reading it, so nothing has to be cleared.  Calls
 *     whose GPU work overlaps (different streams, or host threads without ordering) race
 *     on the array: order them on one stream. */
#define RWKV_NOALLOC_SCRATCH_BYTES (4u << 20)
int rwkv_wkv6_forward_bf16_noalloc(int64_t B, int64_t T, int64_t H, int64_t N,
                                   const uint16_t *r, const uint16_t *k, const uint16_t *v,
                                   const uint16_t *w, const float *u, const float *s0,
                                   uint16_t *y, float *sT, int segments);

/* Test hook for the failure path (process-wide).  While enabled, every chunked WKV-6 forward
 * kernel, every kernel of the chunked delta rule (forward and backward) and both kernels of
 * the state pools wait, before they compute or move anything, on a barrier that nothing
 * signals, with a short bound; the wait runs out, the kernel records RWKV_ERR_TIMEOUT in the
 * device status word, releases its resources and returns (outputs are then unspecified).  No
 * fault or hang is involved.  Returns the previous setting. */
int rwkv_debug_inject_timeout(int enable);

/* ------------------------------------------------------------------ runtime plumbing */
/* Stream used by launches from the calling thread (a cudaStream_t; NULL = legacy
 * default stream).  Thread-local; the caller keeps the stream alive. */
void rwkv_set_stream(void *cuda_stream);
void *rwkv_get_stream(void);

/* Synchronises the calling thread's stream, then returns and clears the device status
 * word of the current device: RWKV_OK, or the first error a kernel recorded since the
 * last call (e.g. RWKV_ERR_TIMEOUT).  Returns RWKV_ERR_CUDA if the synchronisation
 * itself fails. */
int rwkv_get_device_status(void);

/* Static description of a status code. */
const char *rwkv_status_string(int status);

/* Thread-local text of the last failing call's error ("" if none). */
const char *rwkv_last_error(void);

/* RWKV_ABI_VERSION of the loaded library. */
int rwkv_abi_version(void);

/* 1 if the loaded library is the bounds-checked debug build (compiled with
 * WKV_DEBUG_BOUNDS), else 0.  In that build every kernel checks its global, shared-memory and
 * tensor-memory indices and TMA coordinates; a failed check skips the access and records
 * RWKV_ERR_BOUNDS in the device status word (rwkv_get_device_status) -- nothing traps.  It
 * is meant for tests on new shapes; it runs slower. */
int rwkv_debug_bounds(void);

#ifdef __cplusplus
}
#endif

#endif /* RWKV_WKV_H */
