/*
 * gdn.h -- C ABI of libgdn.so: the Gated DeltaNet forward on one NVIDIA
 * GB300 (sm_103a), chunk-wise parallel prefill and single-token decode step.
 *
 * Sources (web pages on Gated DeltaNet):
 *  [Lab3]  "Lab3 GDN Prefill" (hpc101.zjusct.io).
 *          Section "Linear Attention 与 Gated DeltaNet": the gated delta rule
 *            S_t = alpha_t (I - beta_t k_t^T k_t) S_{t-1} + beta_t k_t^T v_t,
 *            o_t = q_t S_t (row vectors; S is dk x dv).
 *          Section "计算过程描述": the chunk form with C = 64,
 *            A = (I + StrictLower(B Gamma K K^T Gamma^-1))^-1,
 *            U = A B V, W = A B Gamma K,
 *            S_[c+1] = gamma_l S_[c] + gamma_l K^T Gamma^-1 (U - W S_[c]),
 *            O_[c] = (1/sqrt dk)[Gamma Q S_[c] + Gamma Lower(Q K^T) Gamma^-1 (U - W S_[c])],
 *            valid chunk length l_c = min(C, L - cC), tail columns masked.
 *          Section "输入输出定义": tensor interface, raw_g = log(alpha) with a
 *            prefix sum restarted at every chunk, optional initial state,
 *            GVA head map h_qk = floor(h_v / (Hv / Hq)).
 *  [SGL]   "sgl-qwen3-5-moe" (rainlin-net), decode node 7
 *          (gdn_packed_recurrent_qk_norm_gating_state_update): one token,
 *          decay -> predict -> correct -> read, state held in f32; its
 *          steps one and two: q/k L2 norm with eps 1e-6 inside the root and
 *          the query scale, gates g = -exp(A_log) softplus(a + dt_bias),
 *          beta = sigmoid(b).
 *  [Kestrel] "Kestrel_VLLM-24 · GDN 线性注意力上 GPU" (wsisp.com), its
 *          CPU-versus-kernel table: softplus with linear / exponential
 *          branches beyond +-20, q/k normalised per k-head before the
 *          v-heads are expanded.
 *
 * Conventions shared by every entry point
 *  - All tensor pointers are DEVICE pointers owned by the caller. The library
 *    never allocates, frees or synchronises; all work is enqueued on `stream`
 *    (a cudaStream_t passed as void*, NULL = the legacy default stream).
 *  - Layouts are contiguous and row-major, token-major:
 *      q, k   [total_tokens, hq, dk]      io_dtype
 *      v, out [total_tokens, hv, dv]      io_dtype
 *      g, beta[total_tokens, hv]          float32 (g is the raw log-decay)
 *      state  [num_seqs or slots, hv, dk, dv] float32
 *    Every pointer must be 16-byte aligned (the per-head gate inputs of
 *    gdn_recurrent_step_gated only 4-byte aligned).
 *  - Supported: dk = dv = 128, chunk size 64 (fixed), hv % hq == 0,
 *    io_dtype GDN_DT_F32 (SIMT f32 arithmetic) or GDN_DT_BF16 (tensor-core
 *    bf16 operands with f32 accumulation and f32 state). Anything else returns
 *    GDN_EUNSUPPORTED without launching.
 *  - Every argument is checked before the first launch; on a non-zero return
 *    nothing was enqueued and no output was touched.
 *  - Checks that need device data (cu_seqlens, state_indices) run on the
 *    device; a failure there is recorded in a device status word (read it with
 *    gdn_read_device_status) and the affected work is skipped.
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gdn_status {
    GDN_OK = 0,
    GDN_EINVAL = 1,        /* bad pointer, shape, size or alignment */
    GDN_EUNSUPPORTED = 2,  /* valid but not implemented (dk/dv != 128, flags) */
    GDN_ECUDA = 3,         /* a CUDA runtime call or launch failed */
    GDN_ETIMEOUT = 4,      /* a bounded device-side wait gave up */
    GDN_EDEVICE_INPUT = 5, /* device-side check failed (cu_seqlens, slot index) */
    GDN_ETOOBIG = 6        /* problem exceeds the fixed scratch of gdn_chunk_fwd_noalloc */
} gdn_status;

typedef enum gdn_dtype {
    GDN_DT_F32 = 0,
    GDN_DT_BF16 = 1
} gdn_dtype;

/* gdn_problem.flags: options of the decode entry points, the precision of
 * [SGL]'s packed decode kernel (node 7). Prefill entry points want 0. */
#define GDN_FLAG_BETA_BF16 (1u << 1)  /* beta rounded to the nearest bf16 (ties to even) before use */
#define GDN_FLAG_STATE_BF16 (1u << 2) /* the state array holds bf16: loaded to f32, the updated state
                                          rounded to bf16 when written back */

/* gdn_problem.flags of the gated linear recurrence (gdn_linear_recurrence and
 * its backward pass and decode step; no other entry point takes it). */
#define GDN_FLAG_GATE_CHANNEL (1u << 3) /* a gate for every channel, [rows, hv, 128] in the io dtype;
                                           without it one per head, [rows, hv] f32 */

/* Problem descriptor.
 *  Dense prefill  : batch = B, seqlen = T, num_seqs = B, total_tokens = B*T,
 *                   cu_seqlens = NULL (sequence b = rows [b*T, (b+1)*T)).
 *  Packed prefill : batch = 1, seqlen = 0, num_seqs = N, total_tokens = rows,
 *                   cu_seqlens = device int32 [N+1].
 *  Decode step    : num_seqs = N tokens (one per sequence), total_tokens = N,
 *                   num_state_slots = rows of the state array.
 */
typedef struct gdn_problem {
    int32_t batch;
    int32_t seqlen;
    int32_t num_seqs;
    int32_t total_tokens;
    int32_t hq;
    int32_t hv;
    int32_t dk;
    int32_t dv;
    int32_t io_dtype;         /* gdn_dtype of q, k, v and out */
    uint32_t flags;           /* GDN_FLAG_* bits (decode only); 0 for prefill */
    int32_t num_state_slots;  /* decode only */
} gdn_problem;

/* Workspace bytes gdn_chunk_fwd needs for problem `p` (0 if `p` is invalid).
 * Sized from an upper bound on the number of 64-token chunks,
 * total_tokens / 64 + num_seqs, so it does not depend on cu_seqlens values. */
size_t gdn_chunk_fwd_workspace_size(const gdn_problem *p);

/* Chunk-wise parallel prefill forward ([Lab3] "计算过程描述").
 *   q, k          [total_tokens, hq, 128]  L2-normalised by the caller
 *   v             [total_tokens, hv, 128]
 *   g             [total_tokens, hv] raw per-token log-decay (log alpha);
 *                 the library does the per-chunk prefix sum
 *   beta          [total_tokens, hv]
 *   scale         multiplies every read-out term (1/sqrt(dk) on the pages)
 *   initial_state [num_seqs, hv, 128, 128] f32, or NULL for zeros
 *   cu_seqlens    int32 [num_seqs+1] packed offsets, or NULL (dense layout).
 *                 Must start at 0, be non-decreasing and end at total_tokens
 *                 (checked on the device). Each sequence starts its own chunk
 *                 grid; chunks never straddle sequences.
 *   out           [total_tokens, hv, 128] written for every token
 *   final_state   [num_seqs, hv, 128, 128] f32, or NULL to skip. A sequence
 *                 of length 0 copies its initial state (or zeros).
 *   workspace     device scratch of at least gdn_chunk_fwd_workspace_size(p)
 *                 bytes, 256-byte aligned; contents need no initialisation
 *                 and are garbage afterwards. Calls that share a workspace
 *                 must be ordered on one stream.
 * Returns GDN_OK once everything is enqueued. */
int gdn_chunk_fwd(const gdn_problem *p, const void *q, const void *k, const void *v,
                  const float *g, const float *beta, float scale,
                  const float *initial_state, const int32_t *cu_seqlens,
                  void *out, float *final_state,
                  void *workspace, size_t workspace_bytes, void *stream);

/* gdn_chunk_fwd followed by the layer's output gate ([SGL] node
 * output_rmsnorm_silu_gate; the gated-RMSNorm row of [Kestrel]): out receives,
 * for every token t and v-head h,
 *   y[t,h] = o[t,h] / sqrt(mean_j o[t,h,j]^2 + norm_eps) * norm_weight * silu(z[t,h])
 * where o is what gdn_chunk_fwd would have written (rounded to the io dtype
 * first, as [SGL]'s node reads it). The other arguments and results are
 * gdn_chunk_fwd's (same workspace size).
 *   z           [total_tokens, hv, 128] io dtype, 16-byte aligned (not NULL)
 *   norm_weight [128] f32, 16-byte aligned; norm_eps >= 0
 * The bf16 path applies the gate inside its fused kernel, on the prepare
 * CTAs once their units are done, tile by tile as the walks finish them; the
 * f32 path runs the gdn_gated_rmsnorm pass after its output kernel. */
int gdn_chunk_fwd_gated(const gdn_problem *p, const void *q, const void *k, const void *v,
                        const float *g, const float *beta, float scale,
                        const float *initial_state, const int32_t *cu_seqlens,
                        const void *z, const float *norm_weight, float norm_eps,
                        void *out, float *final_state,
                        void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of the static device scratch array behind gdn_chunk_fwd_noalloc. */
#define GDN_NOALLOC_SCRATCH_BYTES (32u << 20)

/* gdn_chunk_fwd for callers that cannot allocate device memory.
 * The method itself has no counterpart of this entry point on the pages; it
 * exists for callers that are not allowed to call cudaMalloc (for example
 * code running inside a memory allocator's own hooks, a host callback, or a
 * runtime that fixes its memory footprint after start-up) and so cannot hand
 * over a workspace. Same arguments and results as gdn_chunk_fwd, minus the
 * workspace: the scratch lives in one file-scope device array of
 * GDN_NOALLOC_SCRATCH_BYTES (32 MiB) that every GPU loading the library holds
 * until the process exits. No call allocates or frees anything.
 *  - Returns GDN_ETOOBIG, without launching, when
 *    gdn_chunk_fwd_workspace_size(p) > GDN_NOALLOC_SCRATCH_BYTES. With the
 *    Qwen3.5-style layer (hq = 16, hv = 32) one sequence fits up to 959
 *    tokens on the bf16 path and 447 on the f32 path (the workspace grows by
 *    about 2.1 MB (bf16) or 4.7 MB (f32) per 64-token chunk at hv = 32;
 *    fewer v-heads fit proportionally more tokens). Larger prefills use
 *    gdn_chunk_fwd with a caller workspace.
 *  - The first call on a device (and the first after a cudaDeviceReset of
 *    it) looks up the array's device address with cudaGetSymbolAddress, with
 *    that device current; later calls reuse the address.
 *  - All calls share the one array and it keeps the last call's contents;
 *    nothing in it needs to start at zero. Calls whose work overlaps on the
 *    GPU (different streams, different host threads without ordering) race
 *    on it: order them on one stream. */
int gdn_chunk_fwd_noalloc(const gdn_problem *p, const void *q, const void *k, const void *v,
                          const float *g, const float *beta, float scale,
                          const float *initial_state, const int32_t *cu_seqlens,
                          void *out, float *final_state, void *stream);

/* Single-token recurrent decode step, state updated in place
 * ([Lab3] gated delta rule; [SGL] decode node 7 operation order).
 * For each sequence n < num_seqs and v-head h, with slot s = state_indices[n]
 * (or n when state_indices is NULL) and alpha = exp(g[n,h]):
 *   S = alpha * state[s,h];  p = k_n S;  d = beta (v_n - p);
 *   state[s,h] = S + k_n^T d;  out[n,h] = scale * q_n state[s,h].
 *   q, k [num_seqs, hq, 128]; v, out [num_seqs, hv, 128]; g, beta [num_seqs, hv]
 *   state [num_state_slots, hv, 128, 128] f32 (bf16 with GDN_FLAG_STATE_BF16),
 *   read and written in place; arithmetic is f32 either way.
 *   p->flags may hold GDN_FLAG_BETA_BF16 and GDN_FLAG_STATE_BF16 (any other
 *   bit: GDN_EUNSUPPORTED).
 *   state_indices int32 [num_seqs] or NULL. A negative index skips the
 *   sequence (its out rows are not written: a padding slot). An index
 *   >= num_state_slots is skipped and recorded as GDN_EDEVICE_INPUT.
 *   Two sequences must not name the same slot (their updates would race). */
int gdn_recurrent_step(const gdn_problem *p, const void *q, const void *k, const void *v,
                       const float *g, const float *beta, float scale,
                       void *state, const int32_t *state_indices,
                       void *out, void *stream);

/* Decode step from the raw projections: gdn_recurrent_step with its
 * front-end fused in (decode node 7 of [SGL], steps one and two; the gating
 * kernel of [Kestrel]). For each sequence n and v-head h (k-head
 * kh = h / (hv / hq)):
 *   k_bar = k[n,kh] / sqrt(sum_j k[n,kh,j]^2 + 1e-6)
 *   q_bar = scale * q[n,kh] / sqrt(sum_j q[n,kh,j]^2 + 1e-6)
 *   g     = -exp(A_log[h]) * softplus(a[n,h] + dt_bias[h]),  alpha = exp(g)
 *   beta  = 1 / (1 + exp(-b[n,h]))
 * where softplus(x) is x above 20, exp(x) below -20, log1p(exp(x)) between.
 * Then, as gdn_recurrent_step with scale 1 on q_bar:
 *   S = alpha * state[s,h];  d = beta (v[n,h] - k_bar S);
 *   state[s,h] = S + k_bar^T d;  out[n,h] = q_bar state[s,h].
 *   q, k      [num_seqs, hq, 128] raw (not normalised), io dtype
 *   v, out    [num_seqs, hv, 128], io dtype
 *   a, b      [num_seqs, hv] f32: the gate projections (a drives the decay,
 *             b the write strength)
 *   A_log, dt_bias [hv] f32: per-head parameters
 *   scale     the query scale, 1/sqrt(128) on the pages; applied once
 *   state, state_indices, flags: as gdn_recurrent_step (in place; negative
 *             index = padding slot, skipped; index >= num_state_slots is
 *             skipped and recorded as GDN_EDEVICE_INPUT).
 * All pointers are caller-owned device memory; q, k, v, out, state and
 * state_indices 16-byte aligned, a, b, A_log, dt_bias 4-byte aligned.
 *   z, norm_weight, norm_eps: optional output gate. With z non-NULL
 *             ([num_seqs, hv, 128] io dtype, 16-byte aligned; norm_weight
 *             [128] f32, 16-byte aligned) out receives
 *             y = o / sqrt(mean(o^2) + norm_eps) * norm_weight * silu(z)
 *             per head, computed from the f32 o (as gdn_gated_rmsnorm, but
 *             without rounding o first); with z NULL out receives o and
 *             norm_weight is ignored.
 * Returns GDN_EINVAL (nothing launched) on a bad descriptor or pointer.
 * beta is used in f32 unless p->flags holds GDN_FLAG_BETA_BF16 (the bf16
 * rounding of [SGL]'s packed kernel). */
int gdn_recurrent_step_gated(const gdn_problem *p, const void *q, const void *k, const void *v,
                             const float *a, const float *b, const float *A_log, const float *dt_bias,
                             float scale, void *state, const int32_t *state_indices,
                             const void *z, const float *norm_weight, float norm_eps,
                             void *out, void *stream);

/* Output gate of the GDN layer ([SGL] node output_rmsnorm_silu_gate; the
 * gated-RMSNorm row of [Kestrel]): for every token t and v-head h,
 *   y[t,h] = o[t,h] / sqrt(mean_j o[t,h,j]^2 + eps) * weight * silu(z[t,h])
 * over the head's 128 channels, normalised before the gate; silu(x) =
 * x / (1 + exp(-x)); the weight multiplies directly.
 *   o, z, y  [total_tokens, hv, 128] io dtype (16-byte aligned); y may be o
 *            (in place)
 *   weight   [128] f32 (16-byte aligned), shared by the heads
 *   eps      the RMSNorm epsilon (the pages leave it symbolic)
 * Only total_tokens, hv, dv and io_dtype of `p` are used (dv must be 128).
 * Returns GDN_EINVAL (nothing launched) on a bad descriptor or pointer. */
int gdn_gated_rmsnorm(const gdn_problem *p, const void *o, const void *z, const float *weight, float eps,
                      void *y, void *stream);

/* Short causal depthwise convolution + SiLU with its state, and the split of
 * its output into q, k, v ([Kestrel] conv+SiLU row: window [s0, s1, s2, x_t]
 * oldest first, the state holding the convolution's inputs; [SGL] node 6:
 * x~[t,c] = SiLU(sum_l w[c,l] x[t-l,c] + b[c]), and its layout step).
 * Channels c < C = (2 hq + hv) * 128, taps K = 4, for every packed token t
 * of sequence n (cu_seqlens) at position p:
 *   y[t,c] = SiLU(bias[c] + sum_j weight[c,j] * e[p + j, c]),  j = 0 .. 3,
 * where e = [state of n (3 rows, oldest first) ; the sequence's inputs x], so
 * weight[c,3] multiplies x[t] and weight[c,0] the input three steps back
 * ([SGL]'s lag-l weight is weight[c, 3 - l]). Then q[t] = y[t, 0 : hq*128),
 * k[t] = y[t, hq*128 : 2*hq*128), v[t] = y[t, 2*hq*128 : C), each as
 * [hq or hv, 128] rows; with norm_qk != 0 each q and k head row is divided
 * by sqrt(its sum of squares + 1e-6) ([SGL] node 7 step one, without the
 * query scale). The state of sequence n becomes the last 3 rows of e (the
 * last three inputs; part of the old state when the sequence is shorter).
 *   x          [total_tokens, C] io dtype, 16-byte aligned
 *   weight     [C, 4] f32, bias [C] f32 or NULL (zero), 16-byte aligned
 *   conv_state [num_state_slots, 3, C] io dtype, read and written in place,
 *              or NULL (zero history, nothing written)
 *   state_indices int32 [num_seqs] or NULL (sequence n uses slot n); a
 *              negative index means zero history and no state write; an
 *              index >= num_state_slots is treated the same and recorded as
 *              GDN_EDEVICE_INPUT
 *   cu_seqlens int32 [num_seqs + 1] packed offsets (checked on the device),
 *              or NULL for one sequence of total_tokens (num_seqs must be 1).
 *              Decode: one token per sequence, cu_seqlens = 0, 1, ..., N.
 *   q, k       [total_tokens, hq, 128], v [total_tokens, hv, 128], io dtype
 * Two sequences must not name the same slot. Returns GDN_EINVAL (nothing
 * launched) on a bad descriptor or pointer. */
int gdn_causal_conv1d_silu(const gdn_problem *p, const void *x, const float *weight, const float *bias,
                           void *conv_state, const int32_t *state_indices, const int32_t *cu_seqlens,
                           int norm_qk, void *q, void *k, void *v, void *stream);

/* gdn_causal_conv1d_silu for one token per sequence (decode): sequence n is
 * token n (total_tokens == num_seqs, no offsets); the same arguments
 * otherwise, with x [num_seqs, C] and q, k, v [num_seqs, h, 128]. Its state
 * moves on by one input: [s1, s2, x]. */
int gdn_causal_conv1d_silu_step(const gdn_problem *p, const void *x, const float *weight, const float *bias,
                                void *conv_state, const int32_t *state_indices, int norm_qk,
                                void *q, void *k, void *v, void *stream);

/* Gates of every token from the gate projections ([SGL] gdn_gating node;
 * [Kestrel] gating kernel, softplus linear above 20 and exponential below
 * -20): for t < total_tokens, h < hv,
 *   g[t,h] = -exp(A_log[h]) * softplus(a[t,h] + dt_bias[h]),
 *   beta[t,h] = 1 / (1 + exp(-b[t,h])),
 * ready for gdn_chunk_fwd (g is the raw per-token log-decay).
 *   a, b, g, beta [total_tokens, hv] f32; A_log, dt_bias [hv] f32; all
 *   4-byte aligned. */
int gdn_gating(const gdn_problem *p, const float *a, const float *b, const float *A_log, const float *dt_bias,
               float *g, float *beta, void *stream);

/* ---- training and long sequences: recurrence, norm, output gate ----
 *
 * An output (workspace and states among them) that overlaps an input or another
 * output is refused with GDN_EINVAL, but for the places where one may be the
 * other, which then have the same first byte. (dweight, dbias and d_weight are
 * written when all inputs have been read: only other outputs count for them.) */

/* Gated linear recurrence, a mixer whose state is one value per channel: for
 * every sequence, in token order, and every head h and channel j,
 *   s[t,h,j] = exp(g[t,h,j]) * s[t-1,h,j] + x[t,h,j],   out[t,h,j] = s[t,h,j],
 * s before the first token being the sequence's initial state. The sequence
 * layout, dense or packed, is gdn_chunk_fwd's. Only batch, seqlen, num_seqs,
 * total_tokens, hv, dv (128), io_dtype and flags of `p` are used.
 *   x, out        [total_tokens, hv, 128] io dtype, 16-byte aligned
 *   g             log-decays, g <= 0 (-inf forgets the state): [total_tokens,
 *                 hv] f32, 4-byte aligned, one per head (gdn_gating's g), or
 *                 with GDN_FLAG_GATE_CHANNEL [total_tokens, hv, 128] io dtype,
 *                 16-byte aligned. A gate above 0 is not refused, but partial
 *                 products of the decays may then overflow where the
 *                 recurrence itself does not.
 *   initial_state [num_seqs, hv, 128] f32, 16-byte aligned, or NULL for zeros
 *   cu_seqlens    int32 [num_seqs + 1] packed offsets, 4-byte aligned, or
 *                 NULL (dense). Checked on the device: offsets that do not
 *                 start at 0, rise and end at total_tokens are recorded as
 *                 GDN_EDEVICE_INPUT and nothing is written.
 *   final_state   [num_seqs, hv, 128] f32, 16-byte aligned, or NULL; a
 *                 sequence without tokens gets its initial state (or zeros)
 *   states        NULL, or f32 storage of gdn_linear_recurrence_states_size(p)
 *                 bytes, 16-byte aligned, that the backward pass reads: s
 *                 before every 64th row of the packed token axis (what it
 *                 holds for a row that starts a sequence is unspecified)
 * The state and all sums are f32; out is rounded once. Decays of gates per head
 * and of f32 gates are exact to a rounding, those of bf16 gates per channel to
 * (2 + |g| / 4) 2^-24: f32 states are off by 6e-7 where they remember 36 tokens
 * and by 4e-6 at 667. Infinities and NaN stay in their sequence and channel (dg
 * of gates per head sums the head's channels); from the token on where it is
 * infinite, a state is infinite or NaN: products of decays that underflow to 0
 * meet it. (The CTAs that share an axis wait for their tiles and for each other,
 * each wait at most 2 s: GDN_ETIMEOUT in the device status. So in the backward
 * pass.) */
int gdn_linear_recurrence(const gdn_problem *p, const void *x, const void *g, const float *initial_state,
                          const int32_t *cu_seqlens, void *out, float *final_state, float *states, void *stream);

/* Bytes of gdn_linear_recurrence's `states` for problem `p` (0 if `p` is
 * invalid): ceil(total_tokens / 64) * hv * 128 floats. */
size_t gdn_linear_recurrence_states_size(const gdn_problem *p);

/* Backward pass of gdn_linear_recurrence. With e the gradient that reaches a
 * token from the tokens after it (dfinal_state at a sequence's last token):
 *   ds[t] = dout[t] + e,  dx[t] = ds[t],
 *   dg[t] = exp(g[t]) * s[t-1] * ds[t]  (with gates per head summed over the
 *           head's channels),  e = exp(g[t]) * ds[t] for token t - 1,
 * and dinitial_state is the e that leaves the first token.
 *   dout, x, dx    [total_tokens, hv, 128] io dtype, 16-byte aligned
 *   g, dg          as gdn_linear_recurrence's g
 *   states         what gdn_linear_recurrence wrote for the same inputs
 *   initial_state  what the forward pass was given (or NULL)
 *   dfinal_state   [num_seqs, hv, 128] f32, 16-byte aligned, or NULL for zeros
 *   dinitial_state [num_seqs, hv, 128] f32, 16-byte aligned, or NULL; a
 *                  sequence without tokens gets its dfinal_state (or zeros)
 * The state is recomputed in f32 from `states` and x, not taken from the
 * rounded out. */
int gdn_linear_recurrence_bwd(const gdn_problem *p, const void *dout, const void *x, const void *g,
                              const float *states, const float *initial_state, const float *dfinal_state,
                              const int32_t *cu_seqlens, void *dx, void *dg, float *dinitial_state, void *stream);

/* Decode step of the gated linear recurrence, one token per sequence: for
 * n < num_seqs with slot i = state_indices[n] (n when NULL),
 *   state[i,h,j] = exp(g[n,h,j]) * state[i,h,j] + x[n,h,j], out[n] = state[i].
 *   x, out [num_seqs, hv, 128] io dtype; g as gdn_linear_recurrence's
 *   state  [num_state_slots, hv, 128] f32, 16-byte aligned, in place
 *   state_indices int32 [num_seqs], 4-byte aligned, or NULL. A negative index
 *   skips the sequence (its out rows stay as they were); one >=
 *   num_state_slots is skipped and recorded as GDN_EDEVICE_INPUT. Two
 *   sequences must not name the same slot.
 * out may be x. */
int gdn_linear_recurrence_step(const gdn_problem *p, const void *x, const void *g, float *state,
                               const int32_t *state_indices, void *out, void *stream);

/* Layer norm over the last dimension: for every row r of x,
 *   y[r,j] = (x[r,j] - mean_r) * rstd_r * weight[j] + bias[j],
 *   rstd_r = 1 / sqrt(mean_j (x[r,j] - mean_r)^2 + eps).
 * Only total_tokens (rows), dv (the row's width, 1 .. 16384, else
 * GDN_EUNSUPPORTED) and io_dtype of `p` are used.
 *   x, y         [total_tokens, dv] io dtype, 16-byte aligned; y may be x
 *   weight, bias [dv] f32, 16-byte aligned, or NULL (1 and 0)
 *   mean, rstd   [total_tokens] f32, 4-byte aligned, or NULL to skip: kept
 *                for the backward pass
 * The statistics are f32: the mean first, then the squares about it; a mean
 * above four deviations is corrected by that of the values about it. (Rows too
 * wide for one CTA are on two that wait for each other's sums, each wait at
 * most 2 s: GDN_ETIMEOUT in the device status. So in the backward pass.) */
int gdn_layernorm(const gdn_problem *p, const void *x, const float *weight, const float *bias, float eps, void *y,
                  float *mean, float *rstd, void *stream);

/* Backward pass of gdn_layernorm, xhat = (x - mean) rstd, u = dy * weight:
 *   dx = rstd * (u - mean_j u - xhat * mean_j (u * xhat)),
 *   dweight[j] = sum_r dy[r,j] xhat[r,j],  dbias[j] = sum_r dy[r,j].
 *   dy, x, dx      [total_tokens, dv] io dtype, 16-byte aligned; dx may be dy
 *                  or x
 *   mean, rstd     [total_tokens] f32 from the forward pass, 4-byte aligned
 *   weight         as in the forward pass (NULL: 1)
 *   dweight, dbias [dv] f32, 16-byte aligned, or NULL to skip; written (not
 *                  added to), with no rows zeros
 *   workspace      gdn_layernorm_bwd_workspace_size(p) bytes, 256-byte
 *                  aligned; may be NULL when dweight and dbias are. Calls that
 *                  share it must be ordered on one stream.
 * The sums over rows are taken in a fixed order: the same call gives the same
 * bits. */
int gdn_layernorm_bwd(const gdn_problem *p, const void *dy, const void *x, const float *mean, const float *rstd,
                      const float *weight, void *dx, float *dweight, float *dbias, void *workspace,
                      size_t workspace_bytes, void *stream);
size_t gdn_layernorm_bwd_workspace_size(const gdn_problem *p);

/* Backward pass of gdn_gated_rmsnorm, per (token, head) row with r =
 * 1 / sqrt(mean_j o_j^2 + eps), n = o r, u = dy * weight * silu(z):
 *   d_o = r * (u - n * mean_j (u * n)),
 *   d_z = dy * n * weight * silu'(z),  silu'(z) = s + z s (1 - s), s = 1 / (1 + exp(-z)),
 *   d_weight[j] = sum over rows of dy * n * silu(z).
 *   dy, o, z, d_o, d_z [total_tokens, hv, 128] io dtype, 16-byte aligned; an
 *                output may be any of the inputs (not the other output)
 *   weight       [128] f32, eps: as in the forward pass
 *   d_weight     [128] f32, 16-byte aligned, or NULL to skip; written (not
 *                added to), with no rows zeros
 *   workspace    gdn_gated_rmsnorm_bwd_workspace_size(p) bytes, 256-byte
 *                aligned; may be NULL when d_weight is. Calls that share it
 *                must be ordered on one stream.
 * The sum over rows is taken in a fixed order. */
int gdn_gated_rmsnorm_bwd(const gdn_problem *p, const void *dy, const void *o, const void *z, const float *weight,
                          float eps, void *d_o, void *d_z, float *d_weight, void *workspace, size_t workspace_bytes,
                          void *stream);
size_t gdn_gated_rmsnorm_bwd_workspace_size(const gdn_problem *p);

/* ---- linear attention with a decay for each head ---- */

/* Over each sequence, per value head h with lambda = exp(decay[h]) and its
 * query and key head floor(h / (hv / hq)):
 *   S_t = lambda S_{t-1} + k_t^T v_t,  o_t = scale q_t S_t   (S is dk x dv)
 * (the recurrence of [Lab3] "Linear Attention 与 Gated DeltaNet" with a
 * constant gate), chunk by chunk as gdn_chunk_fwd. Layouts, packed and dense,
 * are gdn_chunk_fwd's.
 *   q, k          [total_tokens, hq, 128] io dtype (used as they are)
 *   v, out        [total_tokens, hv, 128] io dtype
 *   decay         [hv] f32, 4-byte aligned: the log of the factor a token's
 *                 state is kept by, <= 0 (0 keeps all, -inf nothing)
 *   initial_state [num_seqs, hv, 128, 128] f32, or NULL for zeros
 *   cu_seqlens    int32 [num_seqs+1], or NULL (dense), checked on the device
 *   final_state   [num_seqs, hv, 128, 128] f32, or NULL to skip. A sequence
 *                 of length 0 copies its initial state (or zeros).
 *   workspace     gdn_linear_attention_workspace_size(p) bytes, 256-byte
 *                 aligned; contents need no initialisation. Calls that share a
 *                 workspace must be ordered on one stream (captured graphs that
 *                 share one, too).
 * States and sums are f32, decays powers taken from their exponent. bf16: the
 * decayed scores inside a chunk of 128 tokens and the state in the product
 * with q are rounded to bf16, as out is; final_state is not rounded on its way
 * (a token's part of it is exact to 2^-24, and the tensor cores cut the sums over
 * a chunk's tokens: 5e-7 of the state's norm as measured, however many chunks).
 * Where a decay from a chunk's start to a token is below 2^-64, it counts as 2^-64
 * in the product of q with the state, and scores q k above 2^63 overflow there.
 * Infinities and NaN stay in their sequence and value heads, and in f32 reach only
 * tokens whose sums they are in. With bf16 those of v also reach out up to 127
 * tokens before their own, and in the backward pass those of k dq as far, those of
 * dout dv and those of q dk up to 127 tokens behind. (The bf16 kernels wait for
 * copies and products, at most 2 s a wait: GDN_ETIMEOUT in the device status.) */
int gdn_linear_attention(const gdn_problem *p, const void *q, const void *k, const void *v, const float *decay,
                         float scale, const float *initial_state, const int32_t *cu_seqlens, void *out,
                         float *final_state, void *workspace, size_t workspace_bytes, void *stream);
size_t gdn_linear_attention_workspace_size(const gdn_problem *p);

/* Backward pass of gdn_linear_attention: with dS_t = scale q_t^T dout_t +
 * lambda dS_{t+1} (behind a sequence's last token dfinal_state, undecayed),
 *   dq_t = scale dout_t S_t^T,  dk_t = v_t dS_t^T,  dv_t = k_t dS_t,
 *   dinitial_state = lambda dS of the first token,
 * dq and dk summed over the value heads of each query and key head in their
 * order. The decays are constants of the model and get no gradient.
 *   dout, dv       [total_tokens, hv, 128] io dtype
 *   dq, dk         [total_tokens, hq, 128] io dtype
 *   initial_state  what the forward pass was given (or NULL)
 *   dfinal_state   [num_seqs, hv, 128, 128] f32, or NULL for zeros
 *   dinitial_state [num_seqs, hv, 128, 128] f32, or NULL to skip; a sequence
 *                  without tokens gets its dfinal_state (or zeros)
 *   workspace      gdn_linear_attention_bwd_workspace_size(p) bytes
 * The states are recomputed from the inputs; precision as in the forward pass.
 * The same call gives the same bits. */
int gdn_linear_attention_bwd(const gdn_problem *p, const void *dout, const void *q, const void *k, const void *v,
                             const float *decay, float scale, const float *initial_state, const float *dfinal_state,
                             const int32_t *cu_seqlens, void *dq, void *dk, void *dv, float *dinitial_state,
                             void *workspace, size_t workspace_bytes, void *stream);
size_t gdn_linear_attention_bwd_workspace_size(const gdn_problem *p);

/* Decode step of linear attention, one token per sequence: for n < num_seqs
 * with slot i = state_indices[n] (n when NULL),
 *   state[i] = lambda state[i] + k_n^T v_n,  out_n = scale q_n state[i].
 *   q, k [num_seqs, hq, 128], v, out [num_seqs, hv, 128] io dtype; decay as above
 *   state [num_state_slots, hv, 128, 128] f32 (bf16 with GDN_FLAG_STATE_BF16:
 *        out is taken from the f32 state, which is then rounded), in place
 *   state_indices int32 [num_seqs] or NULL. A negative index skips the sequence
 *        (its out rows stay as they were); one >= num_state_slots is skipped and
 *        recorded as GDN_EDEVICE_INPUT. Two sequences must not name the same slot. */
int gdn_linear_attention_step(const gdn_problem *p, const void *q, const void *k, const void *v, const float *decay,
                              float scale, void *state, const int32_t *state_indices, void *out, void *stream);

/* ---- norm and rotation of queries and keys ---- */

/* Descriptor of gdn_qk_norm_rope and its backward pass. Strides are elements
 * from a token to the next, a multiple of 16 bytes and at least the heads'
 * elements: a token's heads lie together, so that slices of a projection's
 * rows need no copy. */
typedef struct gdn_qk_rope {
    int32_t tokens, hq, hk;
    int32_t rotary;              /* channels rotated, the first ones of a head: even, 0 .. 128 */
    int32_t axes;                /* 1 .. 8 */
    int32_t interleaved;         /* pairs: 0: channels (i, i + rotary / 2); 1: (2 i, 2 i + 1) */
    int32_t io_dtype;            /* gdn_dtype of q, k, the outputs and their gradients */
    float eps;
    int64_t q_stride, k_stride;
    int64_t out_q_stride, out_k_stride;   /* of out_q and out_k; backward: of dq and dk */
    int64_t dout_q_stride, dout_k_stride; /* backward only */
} gdn_qk_rope;

/* The norm of every query and key head and its rotation by position: with
 * n = x / sqrt(mean_j x_j^2 + eps) * weight and t = position * inv_freq,
 *   (y_a, y_b) = (n_a cos t - n_b sin t, n_a sin t + n_b cos t)
 * for every pair (a, b); channels behind `rotary` are n. With several axes
 * (time, height, width of a patch) each pair is turned by the position of its
 * own axis.
 *   q, out_q      [tokens, hq, 128] io dtype, 16-byte aligned; k and out_k with
 *                 hk heads; out_q may be q and out_k may be k, in exactly their
 *                 places
 *   q_weight, k_weight [128] f32, 4-byte aligned, or NULL (1)
 *   inv_freq      [rotary / 2] f32: radians per position of each pair
 *   positions     int32 [axes, tokens]
 *   pair_axis     int32 [rotary / 2], the axis that turns a pair, or NULL (axis 0)
 * The angle's error is below 2^-22 radian for every int32 position and
 * frequencies up to 64, all else is f32 and rounded once (a row whose mean square
 * overflows f32 counts as one of infinite norm: zeros). An axis outside
 * 0 .. axes - 1 is recorded as GDN_EDEVICE_INPUT and nothing is written. */
int gdn_qk_norm_rope(const gdn_qk_rope *r, const void *q, const void *k, const float *q_weight, const float *k_weight,
                     const float *inv_freq, const int32_t *positions, const int32_t *pair_axis, void *out_q, void *out_k,
                     void *stream);

/* Backward pass of gdn_qk_norm_rope: with dn the outputs' gradient turned back,
 * xhat = x / sqrt(mean x^2 + eps) and u = dn * weight,
 *   dx = (u - xhat mean_j(u xhat)) / sqrt(mean x^2 + eps),
 *   dweight[j] = sum over tokens and heads of dn xhat.
 *   dout_q, dout_k, dq, dk  like q and k; dq may be q or dout_q, dk may be k
 *                 or dout_k
 *   dq_weight, dk_weight [128] f32, or NULL to skip; written (not added to),
 *                 with no tokens zeros
 *   workspace     gdn_qk_norm_rope_bwd_workspace_size(r) bytes, 256-byte
 *                 aligned; may be NULL when both are. Calls that share it must
 *                 be ordered on one stream.
 * The sums over rows are taken in a fixed order. After an axis outside 0 ..
 * axes - 1 (GDN_EDEVICE_INPUT) dq and dk are not written, and the weights'
 * gradients are zeros. */
int gdn_qk_norm_rope_bwd(const gdn_qk_rope *r, const void *dout_q, const void *dout_k, const void *q, const void *k,
                         const float *q_weight, const float *k_weight, const float *inv_freq, const int32_t *positions,
                         const int32_t *pair_axis, void *dq, void *dk, float *dq_weight, float *dk_weight,
                         void *workspace, size_t workspace_bytes, void *stream);
size_t gdn_qk_norm_rope_bwd_workspace_size(const gdn_qk_rope *r);

/* Synchronises `stream`, returns the device status word (GDN_OK or the first
 * device-side error recorded since the last clear) and clears it when
 * `clear` is non-zero. Returns GDN_ECUDA if the CUDA calls themselves fail. */
int gdn_read_device_status(void *stream, int clear);

/* The status read under the name the library's boundary was specified with:
 * gdn_read_device_status(stream, 1). Synchronises `stream`, returns the first
 * device-side error (GDN_ETIMEOUT, GDN_EDEVICE_INPUT) recorded since the last
 * read, or GDN_OK, and resets the word, the way cudaGetLastError resets the
 * runtime's last error. Returns GDN_ECUDA if the CUDA calls themselves fail. */
int gdn_get_device_status(void *stream);

/* Static, human-readable name of a gdn_status value. */
const char *gdn_status_string(int status);

/* Library ABI version (major * 100 + minor). */
int gdn_version(void);

/* ---- measurement hooks (not part of the method; used by benchmarks) ---- */

/* Kernels the library launches, as indices of the gdn_profile_collect arrays. */
typedef enum gdn_kernel {
    GDN_K_CHUNK_TABLE = 0,        /* chunk table from cu_seqlens */
    GDN_K_PREP_SIMT = 1,          /* f32: gate cumsum + KK^T solve + W, U */
    GDN_K_STATE_SIMT = 2,         /* f32: sequential state pass */
    GDN_K_OUTPUT_SIMT = 3,        /* f32: chunk output */
    GDN_K_RECURRENT_STEP = 4,     /* decode step */
    GDN_K_CHUNK_FUSED_TC = 5,     /* bf16: chunk preparation and state walk, one co-resident grid (tensor cores) */
    GDN_K_RECURRENT_STEP_GATED = 6, /* decode step with the gate / q-k norm front-end */
    GDN_K_GATED_RMSNORM = 7,      /* output gate (head-wise RMSNorm, SiLU(z)) over a whole tensor */
    GDN_K_CONV1D_SILU = 8,        /* short causal convolution + SiLU with conv state, split into q, k, v */
    GDN_K_GATING = 9,             /* g and beta from the gate projections, every token */
    GDN_K_CONV1D_STEP = 10,       /* short convolution, one token per sequence (decode) */
    GDN_K_LINREC = 11,            /* gated linear recurrence, forward */
    GDN_K_LINREC_BWD = 12,        /* gated linear recurrence, backward */
    GDN_K_LINREC_STEP = 13,       /* gated linear recurrence, decode step */
    GDN_K_LAYERNORM = 14,         /* layer norm */
    GDN_K_LAYERNORM_BWD = 15,     /* layer norm, backward: dx and partial sums over rows */
    GDN_K_GATED_RMSNORM_BWD = 16, /* output gate, backward: d_o, d_z and partial sums over rows */
    GDN_K_ROW_SUMS = 17,          /* partial sums over rows -> weight and bias gradients */
    GDN_K_LINATTN_TABLE = 18,     /* linear attention: segments of the sequences */
    GDN_K_LINATTN_SUM = 19,       /* linear attention: sums of the segments */
    GDN_K_LINATTN_CHAIN = 20,     /* linear attention: states that enter the segments */
    GDN_K_LINATTN_WALK = 21,      /* linear attention: outputs (gradients) and final states */
    GDN_K_LINATTN_GROUP_SUM = 22, /* linear attention, backward: dq and dk over the heads of a group */
    GDN_K_LINATTN_STEP = 23,      /* linear attention, decode step */
    GDN_K_QK_NORM_ROPE = 24,      /* norm and rotation of queries and keys */
    GDN_K_QK_NORM_ROPE_BWD = 25,  /* its backward pass */
    GDN_K_COUNT = 26
} gdn_kernel;

/* Turns per-kernel CUDA-event timing on (non-zero) or off for every later
 * launch (process-wide). Launch counting is always on. */
int gdn_profile_enable(int enable);

/* Synchronises the recorded events and copies, for the first `count` kernel
 * ids, the number of launches, the summed event time in ms and the number of
 * timed launches into the caller's host arrays (any may be NULL). Clears all
 * counters when `reset` is non-zero. */
int gdn_profile_collect(long long *launches, double *ms, long long *timed, int count, int reset);

/* Static name of a gdn_kernel id. */
const char *gdn_kernel_name(int kernel);

/* Sets, process-wide, the limit of every bounded device-side wait in the
 * kernels launched after the call (the tensor-core prefill kernel's copy, MMA
 * and ready-flag waits; the recurrence's waits on copies and on the other CTAs
 * of a cluster; the layer norm's on the other CTA of a pair; linear attention's
 * on copies and products, counted in cycles of which there is more than one a
 * nanosecond), in nanoseconds of wall time; 0 restores the default of 2 s. A
 * wait that runs out records GDN_ETIMEOUT in the device status word; the kernel
 * then drains what it has in flight (copies, MMAs and stores between CTAs, each
 * drain bounded too), frees its tensor memory and returns, so the context stays
 * usable and the call's outputs are unspecified. Meant for tests of that path:
 * a limit of a few microseconds makes the prefill's waits on not-yet-prepared
 * chunks run out, one of some nanoseconds the others. Returns GDN_OK. */
int gdn_set_wait_limit_ns(unsigned long long ns);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H_ */
