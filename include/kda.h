/*
 * kda.h — C ABI of the MI355X (gfx950) Kimi Delta Attention chunked operator:
 * a forward pass and a backward pass that recomputes its intermediates
 * instead of saving them.
 *
 * Operator ("KDA Memory with Recompute: FLA vs cuDNN Frontend FROST",
 * section "Sources and measurement configuration"; per-chunk operations in
 * "KDA at the production shape..." section 2.1 and section 1.1):
 *   per packed sequence and head, with the state S (K x V) starting at zero,
 *     qh = scale * q / sqrt(|q|^2 + eps),  kh = k / sqrt(|k|^2 + eps)
 *     beta = sigmoid(raw_beta)
 *     g = L * sigmoid(exp(A_log[h]) * (raw_g + dt_bias[h,:]))   (L = gate_lower_bound;
 *         the default gate map, see gate_mode below)
 *     S_t = (I - beta_t kh_t kh_t^T) Diag(exp(g_t)) S_{t-1} + beta_t kh_t v_t^T
 *     o_t = S_t^T qh_t
 *   the state restarts at every sequence boundary of cu_seqlens, from zero
 *   (the measured setting of the FROST page: no initial state, no final
 *   state). The backward returns the gradients of all seven inputs (q, k, v,
 *   raw_g, raw_beta, A_log, dt_bias) of sum(o * dO). kda_fwd_ex / kda_bwd_ex
 *   add an optional initial state per sequence, its final state and their
 *   gradients, and optional forward-saved checkpoints (FROST's
 *   checkpoint_every_n_tokens, same page, "Both sides really use
 *   recomputation").
 *
 * Conventions for every entry point:
 *   - Tensor pointers are DEVICE pointers owned by the caller, row-major with
 *     the innermost dimension contiguous: q, k, raw_g [T, H, K]; v, o, dO
 *     [T, H, V]; raw_beta [T, H]; A_log [H] (fp32); dt_bias [H, K] (fp32)
 *     (raw_g [T, H] and dt_bias [H] under KDA_GATE_PER_HEAD);
 *     cu_seqlens [n_seqs + 1] (int32, device copy). Pointers must be 16-byte
 *     aligned.
 *   - dtype selects the element type of q, k, v, raw_g, raw_beta, dO, o and
 *     of dq, dk, dv, draw_g, draw_beta (fp32 or bf16). dA_log and ddt_bias
 *     are always fp32.
 *   - `stream` is a hipStream_t (passed as void*; NULL is the null stream).
 *     All work is enqueued on it asynchronously; no call synchronises the
 *     host with the device. Outputs are overwritten, never accumulated.
 *   - The library allocates no device memory and keeps no state between
 *     calls: scratch comes from the caller's `workspace` (size from the
 *     *_workspace_bytes query for the same problem). Calls are reentrant and
 *     thread-safe; calls sharing a workspace must be stream-ordered.
 *   - All argument validation happens on the host before any HIP call.
 *     Return value: KDA_OK or one of the error codes below. NaN/Inf inputs
 *     propagate; they are not checked.
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
  KDA_OK = 0,
  KDA_ERR_INVALID = 1,     /* null pointer, non-positive size, bad cu_seqlens_host */
  KDA_ERR_UNSUPPORTED = 2, /* K/V/chunk/dtype/gate combination not built */
  KDA_ERR_WORKSPACE = 3,   /* workspace smaller than the *_workspace_bytes query */
  KDA_ERR_HIP = 4          /* a HIP launch failed; kda_status_string names it */
};

enum { KDA_F32 = 0, KDA_BF16 = 1 };

/* Gate maps (the pages fix the bound L and the FP32 A_log / dt_bias drive,
   not the formula), with z = raw_g + dt_bias[h,:]:
     KDA_GATE_SIGMOID_BOUND   g = L * sigmoid(exp(A_log[h]) * z)
     KDA_GATE_SOFTPLUS_CLAMP  g = max(L, -exp(A_log[h]) * softplus(z));
                              no gradient flows where the bound holds.
   Either may be OR-ed with KDA_GATE_PER_HEAD: one scalar gate per head and
   token, the Gated DeltaNet form of FLA's chunk_gdn ("KDA at the production
   shape...", sections 1.1 and 1.2; KDA adds a decay per key channel). Then
   raw_g and draw_g are [T, H], dt_bias and ddt_bias are [H], z = raw_g[t,h]
   + dt_bias[h], and every channel of the state decays by the same exp(g).
   Other values: KDA_ERR_UNSUPPORTED. */
enum { KDA_GATE_SIGMOID_BOUND = 0, KDA_GATE_SOFTPLUS_CLAMP = 1, KDA_GATE_PER_HEAD = 16 };

typedef struct {
  int32_t n_seqs;          /* N >= 1 packed sequences (empty sequences allowed) */
  int64_t total_tokens;    /* T = cu_seqlens_host[N] >= 1 */
  int32_t H, K, V;         /* heads, key dim, value dim; built: K == V in {64, 128} */
  int32_t chunk;           /* chunk length C; tiling only, the result does not
                              depend on it beyond rounding. Built: fp32 K=64:
                              16, 32, 64; fp32 K=128: 16, 32; bf16 K=64 or
                              128: 32, 64 (others: KDA_ERR_UNSUPPORTED) */
  int32_t dtype;           /* KDA_F32 or KDA_BF16 */
  int32_t gate_mode;       /* KDA_GATE_SIGMOID_BOUND or KDA_GATE_SOFTPLUS_CLAMP,
                              optionally | KDA_GATE_PER_HEAD */
  float scale;             /* multiplies qh; 1.0 for the plain o_t = S_t^T qh_t */
  float gate_lower_bound;  /* L, -5.9 <= L < 0 (e.g. -5). The kernels split
                              every decay exp(G_r - G_s) of a chunk around
                              the first row of a 16-row block, so a factor
                              reaches exp(15 |L|), which must stay finite in
                              fp32 for either dtype: L < -5.9 returns
                              KDA_ERR_UNSUPPORTED, L >= 0 or not finite
                              KDA_ERR_INVALID */
  float l2_eps;            /* eps of the Q/K L2 normalisation, e.g. 1e-6 */
  int32_t seg_chunks;      /* most chunks one streaming segment holds (forward
                              and backward); 0 = automatic (the segments fit
                              the workspace budget). A segment is either a
                              run of the chunk order (sequences one after
                              another) or, for a packed batch with several
                              long sequences, a window of the same chunk
                              positions in every sequence; the library takes
                              the plan whose scans have the shorter chain */
  const int32_t *cu_seqlens_host; /* host copy of cu_seqlens [N+1]: non-decreasing
                                     from 0 to T; used for planning only */
} kda_problem;

/* Bytes of device workspace kda_fwd / kda_bwd need for this problem
   (0 when the problem is invalid or unsupported; call kda_check_problem for
   the reason). */
size_t kda_fwd_workspace_bytes(const kda_problem *p);
size_t kda_bwd_workspace_bytes(const kda_problem *p);

/* Host-side validation only: KDA_OK, KDA_ERR_INVALID or KDA_ERR_UNSUPPORTED. */
int kda_check_problem(const kda_problem *p);

/* Prologue only (the step that normalises Q/K, applies the beta sigmoid,
   the bounded gate and its chunk-local cumulative sum), exposed for testing.
   Outputs, all fp32 and caller-owned: qh, kh [T,H,K]; beta [T,H];
   gcum [T,H,K] = cumulative sum of g from the start of each chunk (chunks
   of length p->chunk counted from each sequence start). The workspace holds
   the chunk table (kda_prologue_workspace_bytes). */
size_t kda_prologue_workspace_bytes(const kda_problem *p);
int kda_prologue(const kda_problem *p, const void *q, const void *k,
                 const void *raw_g, const void *raw_beta, const float *A_log,
                 const float *dt_bias, const int32_t *cu_seqlens, float *qh,
                 float *kh, float *beta, float *gcum, void *workspace,
                 size_t workspace_bytes, void *stream);

/* Forward ("KDA Memory with Recompute: FLA vs cuDNN Frontend FROST", section
   "Sources and measurement configuration": the inputs, the in-kernel
   normalisation, sigmoid and safe gate, packed sequences; "KDA at the
   production shape...", section 2.1, the per-chunk operations, and section
   1.1, the state loop): writes o [T,H,V] (dtype). Saves nothing for the
   backward. Errors: KDA_ERR_INVALID / KDA_ERR_UNSUPPORTED from the problem
   (as kda_check_problem) or a null pointer, KDA_ERR_WORKSPACE when
   workspace_bytes < kda_fwd_workspace_bytes, KDA_ERR_HIP on a failed
   launch; all but the last are found before any launch. */
int kda_fwd(const kda_problem *p, const void *q, const void *k, const void *v,
            const void *raw_g, const void *raw_beta, const float *A_log,
            const float *dt_bias, const int32_t *cu_seqlens, void *o,
            void *workspace, size_t workspace_bytes, void *stream);

/* Backward (the FROST page, sections "Both sides really use recomputation"
   and "Why the larger FROST state series still wins": recompute instead of
   saving, gradients written once in the input dtype; all seven inputs
   differentiated as in "Sources and measurement configuration"):
   recomputes every intermediate from the inputs, streaming over
   segments of chunks, and writes dq, dk, draw_g [T,H,K], dv [T,H,V],
   draw_beta [T,H] (dtype) and dA_log [H], ddt_bias [H,K] (fp32); draw_g
   [T,H] and ddt_bias [H] under KDA_GATE_PER_HEAD. The
   gate-parameter gradients are reduced in a fixed order (bitwise
   reproducible run to run). Errors as kda_fwd, with
   kda_bwd_workspace_bytes. */
int kda_bwd(const kda_problem *p, const void *q, const void *k, const void *v,
            const void *raw_g, const void *raw_beta, const float *A_log,
            const float *dt_bias, const int32_t *cu_seqlens, const void *dO,
            void *dq, void *dk, void *dv, void *draw_g, void *draw_beta,
            float *dA_log, float *ddt_bias, void *workspace,
            size_t workspace_bytes, void *stream);

/* State ends and forward-saved checkpoints (all fp32, device, caller-owned;
   every pointer may be NULL):
     h0    [N, H, K, V]  state each sequence starts from (NULL: zero). An
                         empty sequence passes it through to ht.
     ht    [N, H, K, V]  kda_fwd_ex: the state after each sequence's last
                         token (NULL: not written).
     dht   [N, H, K, V]  kda_bwd_ex: gradient of the loss with respect to ht
                         (NULL: zero), so the gradients are those of
                         sum(o * dO) + sum(ht * dht).
     dh0   [N, H, K, V]  kda_bwd_ex: gradient with respect to h0 (NULL: not
                         written).
     ckpt, ckpt_bytes    kda_fwd_ex writes, kda_bwd_ex reads, the states
                         that enter the backward's segments inside each
                         sequence (kda_checkpoint_bytes bytes, a layout
                         private to the library), so the backward skips the
                         pass that recomputes them. Pass the same problem to
                         both calls (set seg_chunks explicitly, or keep the
                         workspace budget unchanged between them).
                         ckpt_bytes smaller than kda_checkpoint_bytes:
                         KDA_ERR_WORKSPACE.
   The backward still recomputes w, u and h of every chunk. kda_fwd_ex reads
   h0 and writes ht and ckpt; kda_bwd_ex reads h0, dht and ckpt (which it
   leaves unchanged) and writes dh0. The same problem and h0 must be passed
   to both. */
typedef struct {
  const float *h0;
  float *ht;
  const float *dht;
  float *dh0;
  float *ckpt;
  size_t ckpt_bytes;
} kda_state_io;

/* Bytes of the checkpoint buffer of kda_state_io for this problem, and the
   backward's segment length: chunks per segment, or chunks of each sequence
   per segment for a plan by windows (0 when the problem is invalid). */
size_t kda_checkpoint_bytes(const kda_problem *p);
int32_t kda_bwd_segment_chunks(const kda_problem *p);

/* kda_fwd / kda_bwd with state ends and checkpoints (io may be NULL, which
   is kda_fwd / kda_bwd). Workspace sizes are those of kda_fwd_workspace_bytes
   / kda_bwd_workspace_bytes. */
int kda_fwd_ex(const kda_problem *p, const void *q, const void *k, const void *v,
               const void *raw_g, const void *raw_beta, const float *A_log,
               const float *dt_bias, const int32_t *cu_seqlens, void *o,
               const kda_state_io *io, void *workspace, size_t workspace_bytes,
               void *stream);
int kda_bwd_ex(const kda_problem *p, const void *q, const void *k, const void *v,
               const void *raw_g, const void *raw_beta, const float *A_log,
               const float *dt_bias, const int32_t *cu_seqlens, const void *dO,
               void *dq, void *dk, void *dv, void *draw_g, void *draw_beta,
               float *dA_log, float *ddt_bias, const kda_state_io *io,
               void *workspace, size_t workspace_bytes, void *stream);

/* GDN-2 ("KDA at the production shape...", section 1.6, and the per-chunk
   operation table of its section 2.1: akk = (b k Gamma)(k / Gamma)^T,
   w = M^-1 (b k Gamma), u = M^-1 (w v)): the gated delta rule with a
   channel-wise erase gate and a channel-wise write gate in place of beta,
     b = sigmoid(raw_b) [K],  w = sigmoid(raw_w) [V]
     S_t = (I - kh_t (b_t * kh_t)^T) Diag(exp(g_t)) S_{t-1} + kh_t (w_t * v_t)^T
     o_t = S_t^T qh_t
   with the prologue, gate maps, packing and layouts of kda_fwd / kda_bwd.
   KDA is the case b = w = beta in every channel. raw_b [T, H, K] and raw_w
   [T, H, V] are in the problem's dtype (device, caller-owned); the backward
   writes draw_b [T, H, K] and draw_w [T, H, V] in that dtype, with dq, dk,
   dv, draw_g, dA_log, ddt_bias as kda_bwd. Workspace sizes are those of
   kda_fwd_workspace_bytes / kda_bwd_workspace_bytes. Not built for GDN-2
   (KDA_ERR_UNSUPPORTED): a gate per head (KDA_GATE_PER_HEAD), and fp32 at
   K = 64 with 64-token chunks. Errors otherwise as kda_fwd / kda_bwd. */
int kda_gdn2_fwd(const kda_problem *p, const void *q, const void *k, const void *v,
                 const void *raw_g, const void *raw_b, const void *raw_w, const float *A_log,
                 const float *dt_bias, const int32_t *cu_seqlens, void *o, void *workspace,
                 size_t workspace_bytes, void *stream);
int kda_gdn2_bwd(const kda_problem *p, const void *q, const void *k, const void *v,
                 const void *raw_g, const void *raw_b, const void *raw_w, const float *A_log,
                 const float *dt_bias, const int32_t *cu_seqlens, const void *dO, void *dq,
                 void *dk, void *dv, void *draw_g, void *draw_b, void *draw_w, float *dA_log,
                 float *ddt_bias, void *workspace, size_t workspace_bytes, void *stream);

/* kda_gdn2_fwd with the states a prompt starts from and leaves for
   kda_gdn2_recurrent: io->h0 and io->ht as for kda_fwd_ex (io may be NULL).
   GDN-2's backward takes no states, so there is nothing to checkpoint:
   io->ckpt other than NULL is KDA_ERR_INVALID. */
int kda_gdn2_fwd_ex(const kda_problem *p, const void *q, const void *k, const void *v,
                    const void *raw_g, const void *raw_b, const void *raw_w, const float *A_log,
                    const float *dt_bias, const int32_t *cu_seqlens, void *o,
                    const kda_state_io *io, void *workspace, size_t workspace_bytes,
                    void *stream);

/* The recurrent form, for decoding: the same operator token by token, each
   sequence starting from a state in the caller's pool and leaving its last
   state there (the h0 and ht of kda_fwd_ex, fp32 [K][V] per head, so a
   state kda_fwd_ex returned can be decoded from). Per sequence and head:
     S~ = Diag(exp(g_t)) S,  u = S~^T (beta_t kh_t)
     S  = S~ + kh_t (beta_t v_t - u)^T,  o_t = S^T qh_t
   with the prologue and gate maps of kda_fwd.
     cu_seqlens     [N+1] (int32, device) or NULL: one token per sequence,
                    N = T. Values are clamped to [0, T]; an empty sequence
                    leaves its state as it is. Rows of o that belong to no
                    sequence (before cu_seqlens[0], from cu_seqlens[N] on)
                    are not written, or zero with zero_rest.
     state_indices  [N] (int32, device) or NULL: the pool slot of each
                    sequence (NULL: slot n, n_slots >= N). At most 65536
                    sequences (KDA_ERR_UNSUPPORTED). A negative one
                    marks a padded sequence: its rows of o are zero and no
                    state is touched. A slot of n_slots or more, or one that
                    an earlier sequence with tokens names too, is an error
                    that the host cannot see: the sequence's rows of o are
                    NaN and no state is touched.
     state          [n_slots, H, K, V] (fp32, device), updated in place. Its
                    addresses must be apart from those of every other tensor
                    of the call (KDA_ERR_INVALID).
   Nothing is read on the host but the problem, so the call can be captured
   into a graph and replayed with other cu_seqlens and slots of the same N
   and T. It needs no workspace. T = 0 or N = 0: nothing is launched.
   q, k, v, raw_g and raw_beta may have rows further apart than H * K, H * V
   or H elements (the *_stride fields, in elements; 0: rows adjacent), as
   slices of one fused projection have; strides of q, k, v and a per-channel
   raw_g are multiples of 16 bytes. Pointers other than those of raw_beta,
   of a per-head raw_g, cu_seqlens and state_indices are 16-byte aligned. */
typedef struct {
  int32_t n_seqs;          /* N >= 0 */
  int64_t total_tokens;    /* T >= 0; N when cu_seqlens is NULL */
  int32_t H, K, V;         /* built: K == V in {64, 128} */
  int32_t dtype;           /* KDA_F32 or KDA_BF16 */
  int32_t gate_mode;       /* as kda_problem */
  float scale;             /* as kda_problem */
  float gate_lower_bound;  /* as kda_problem */
  float l2_eps;            /* as kda_problem */
  int64_t n_slots;         /* states in the pool */
  int64_t q_stride, k_stride, v_stride; /* elements between tokens; 0: H*K, H*K, H*V */
  int64_t g_stride;        /* 0: H*K, or H under KDA_GATE_PER_HEAD */
  int64_t beta_stride;     /* 0: H (kda_recurrent) */
  int64_t b_stride, w_stride; /* 0: H*K, H*V (kda_gdn2_recurrent) */
  int32_t zero_rest;       /* not 0: zero the rows of o that belong to no sequence */
} kda_recurrent_problem;

/* Errors: KDA_ERR_INVALID (negative or inconsistent sizes, a stride shorter
   than a row or not a multiple of 16 bytes, a null pointer, a state that
   overlaps another tensor), KDA_ERR_UNSUPPORTED (size, dtype or gate not
   built; N * H of 2^24 or more, of 2^24 - 1 with zero_rest), KDA_ERR_HIP. */
int kda_recurrent(const kda_recurrent_problem *p, const void *q, const void *k, const void *v,
                  const void *raw_g, const void *raw_beta, const float *A_log,
                  const float *dt_bias, const int32_t *cu_seqlens,
                  const int32_t *state_indices, float *state, void *o, void *stream);

/* GDN-2's recurrent form (erase gate raw_b [T, H, K], write gate raw_w
   [T, H, V]): u = S~^T (b_t * kh_t), S = S~ + kh_t (w_t * v_t - u)^T, the
   rest as kda_recurrent. KDA_GATE_PER_HEAD is not built for GDN-2. */
int kda_gdn2_recurrent(const kda_recurrent_problem *p, const void *q, const void *k,
                       const void *v, const void *raw_g, const void *raw_b, const void *raw_w,
                       const float *A_log, const float *dt_bias, const int32_t *cu_seqlens,
                       const int32_t *state_indices, float *state, void *o, void *stream);

/* Activations of the gates and of the short convolution. */
enum { KDA_ACT_NONE = 0, KDA_ACT_SIGMOID = 1, KDA_ACT_SILU = 2 };

/* The norm behind the operator, with the output gate: for each row (one
   head of one token)
     y = o / sqrt(mean(o^2) + eps) * weight * act(gate)
   o, gate, y [rows, V] (dtype, rows = T * H), weight [V] (fp32, shared by
   the heads). act is KDA_ACT_SIGMOID or KDA_ACT_SILU. The backward
   recomputes the norm from o and writes d_o, dgate [rows, V] (dtype) and
   dweight [V] (fp32, summed in a fixed order). Pointers are 16-byte aligned;
   outputs must not overlap inputs. rows = 0: nothing but dweight (zero) is
   written. Errors: KDA_ERR_INVALID, KDA_ERR_UNSUPPORTED, KDA_ERR_WORKSPACE
   (backward), KDA_ERR_HIP. */
typedef struct {
  int64_t rows;       /* >= 0 */
  int32_t V;          /* built: 64, 128, 256 */
  int32_t dtype;      /* KDA_F32 or KDA_BF16 */
  int32_t activation; /* KDA_ACT_SIGMOID or KDA_ACT_SILU */
  float eps;          /* >= 0 */
} kda_gated_norm_problem;
int kda_gated_norm_fwd(const kda_gated_norm_problem *p, const void *o, const void *gate,
                       const float *weight, void *y, void *stream);
size_t kda_gated_norm_bwd_workspace_bytes(const kda_gated_norm_problem *p);
int kda_gated_norm_bwd(const kda_gated_norm_problem *p, const void *o, const void *gate,
                       const float *weight, const void *dy, void *d_o, void *dgate,
                       float *dweight, void *workspace, size_t workspace_bytes, void *stream);

/* Between two blocks: the norm after one block's output y, its gate, the
   residual scale, the residual stream x and the norm before the next block.
   For each token
     z = y / sqrt(mean(y^2) + eps) * w_post     (w_post NULL: z = y)
     x_out = x + residual_scale * sigmoid(raw_gate) * z   (no gate: factor 1)
     h = x_out / sqrt(mean(x_out^2) + eps) * w_pre
   x, y, x_out, h [tokens, D] (dtype); w_post, w_pre [D] (fp32); raw_gate
   (dtype) [tokens] (KDA_BLOCK_GATE_TOKEN) or [tokens, D]
   (KDA_BLOCK_GATE_CHANNEL), NULL with KDA_BLOCK_GATE_NONE. h is formed from
   x_out before its rounding to the dtype. The backward recomputes x_out and
   both norms from x, y and raw_gate, takes the gradients dx_out and dh
   (either may be NULL: zero) and writes dx, dy, dgate (dtype) and dw_post,
   dw_pre [D] (fp32, summed in a fixed order). Pointers are 16-byte aligned
   (a per-token gate and its gradient: aligned to their type); outputs must
   not overlap inputs. tokens = 0: nothing but dw_post and dw_pre (zero) is
   written. Errors as for the gated norm. */
enum { KDA_BLOCK_GATE_NONE = 0, KDA_BLOCK_GATE_TOKEN = 1, KDA_BLOCK_GATE_CHANNEL = 2 };
typedef struct {
  int64_t tokens;       /* >= 0 */
  int32_t D;            /* built: multiples of 8 up to 8192 */
  int32_t dtype;        /* KDA_F32 or KDA_BF16 */
  int32_t gate;         /* KDA_BLOCK_GATE_* */
  float residual_scale; /* finite */
  float eps;            /* >= 0 */
} kda_block_norm_problem;
int kda_block_norm_fwd(const kda_block_norm_problem *p, const void *x, const void *y,
                       const void *raw_gate, const float *w_post, const float *w_pre,
                       void *x_out, void *h, void *stream);
size_t kda_block_norm_bwd_workspace_bytes(const kda_block_norm_problem *p);
int kda_block_norm_bwd(const kda_block_norm_problem *p, const void *x, const void *y,
                       const void *raw_gate, const float *w_post, const float *w_pre,
                       const void *dx_out, const void *dh, void *dx, void *dy, void *dgate,
                       float *dw_post, float *dw_pre, void *workspace, size_t workspace_bytes,
                       void *stream);

/* The short causal convolution in front of the operator: depthwise over the
   channels of each packed sequence, W taps, with an activation. With the rows
   e_0 .. e_{W-2} of the sequence's initial state followed by its tokens
   e_{W-1+t} = x_t,
     y_t[c] = act(bias[c] + sum_j weight[c][j] e_{t+j}[c]),  j = 0 .. W-1
   and the final state the last W-1 rows of e (of an empty or short sequence
   some of them rows of its initial state).
     x, y            [T, C] (dtype); x may have rows further apart (x_stride)
     weight, bias    [C, W], [C] (fp32); bias NULL: zero
     cu_seqlens      [N+1] (int32, device), or NULL: one sequence, N = 1.
                     Values are clamped to [0, T]; rows of y (and dx) that
                     belong to no sequence are zero
     initial_state, final_state  [N, W-1, C] (dtype); NULL: zero, not written
   The backward recomputes the activations' inputs, takes dy and d_final_state
   (NULL: zero), and writes dx [T, C] (rows adjacent), d_initial_state (NULL:
   not written) and dweight, dbias (fp32, summed in a fixed order; dbias NULL:
   not written). Pointers are 16-byte aligned (cu_seqlens: 4); outputs must
   not overlap inputs. T = 0 is allowed. Errors: KDA_ERR_INVALID,
   KDA_ERR_UNSUPPORTED, KDA_ERR_WORKSPACE (backward), KDA_ERR_HIP. */
typedef struct {
  int32_t n_seqs;       /* N >= 0; 1 (update: T) when cu_seqlens is NULL */
  int64_t total_tokens; /* T >= 0 */
  int32_t C;            /* built: multiples of 8 up to 2^20 */
  int32_t W;            /* built: 2, 3, 4 */
  int32_t dtype;        /* KDA_F32 or KDA_BF16 */
  int32_t activation;   /* KDA_ACT_NONE or KDA_ACT_SILU */
  int64_t n_slots;      /* update: states in the pool */
  int64_t x_stride;     /* elements between tokens of x, a multiple of 16
                           bytes; 0: C */
  int32_t zero_rest;    /* update, not 0: zero the rows of y that belong to no
                           sequence (the packed form always does) */
} kda_short_conv_problem;
int kda_short_conv_fwd(const kda_short_conv_problem *p, const void *x, const float *weight,
                       const float *bias, const int32_t *cu_seqlens, const void *initial_state,
                       void *y, void *final_state, void *stream);
size_t kda_short_conv_bwd_workspace_bytes(const kda_short_conv_problem *p);
int kda_short_conv_bwd(const kda_short_conv_problem *p, const void *x, const float *weight,
                       const float *bias, const int32_t *cu_seqlens, const void *initial_state,
                       const void *dy, const void *d_final_state, void *dx, float *dweight,
                       float *dbias, void *d_initial_state, void *workspace,
                       size_t workspace_bytes, void *stream);

/* The convolution's decoding form: sequence n starts from its state in a
   pool [n_slots, W-1, C] (dtype) and leaves its last W-1 rows there.
   cu_seqlens, state_indices, padded sequences, rows that belong to no
   sequence, overlap with the state and capture as for kda_recurrent. */
int kda_short_conv_update(const kda_short_conv_problem *p, const void *x, const float *weight,
                          const float *bias, const int32_t *cu_seqlens,
                          const int32_t *state_indices, void *state, void *y, void *stream);

/* For callers that cannot allocate device memory (code under HIP graph
   capture, tight serving loops, harnesses that forbid hipMalloc): kda_fwd
   with its workspace in a device array of KDA_NOALLOC_SCRATCH_BYTES that the
   library holds on each GPU it runs on until the process ends (the caller
   passes inputs and outputs only; layouts and result as kda_fwd, O
   bit-identical to it). The call runs the forward over the longest segment
   of chunks whose workspace fits the array; a problem whose one-chunk
   segment needs more (its state carry slots are 2 * H * K * V * 4 bytes)
   returns KDA_ERR_WORKSPACE. It allocates nothing. Calls on one GPU share
   the array: calls that overlap in time race and must be ordered by the
   caller. Returns KDA_ERR_HIP if the array's device address cannot be
   obtained. */
#define KDA_NOALLOC_SCRATCH_BYTES (64u << 20)
int kda_fwd_noalloc(const kda_problem *p, const void *q, const void *k, const void *v,
                    const void *raw_g, const void *raw_beta, const float *A_log,
                    const float *dt_bias, const int32_t *cu_seqlens, void *o, void *stream);

/* Optional per-kernel timing, for measurement tools. Between
   kda_profile_begin() and kda_profile_end(), every kernel the calling thread
   launches through this library is bracketed by two HIP events recorded on
   its own stream. kda_profile_end() waits for those events and writes, per
   kernel kind (index = KDA_KERNEL_*), the number of launches, their summed
   duration in milliseconds and the summed number of (chunk, head) units the
   launches processed into `launches` / `total_ms` / `units` (arrays of `n`
   entries, caller-owned, each may be NULL; n >= KDA_KERNEL_COUNT
   recommended). Returns KDA_OK or KDA_ERR_HIP. Timing adds two event
   records per launch. */
enum {
  KDA_KERNEL_CHUNK_TABLE = 0,
  KDA_KERNEL_PROLOGUE = 1,
  KDA_KERNEL_CHUNK_LOCAL = 2,       /* forward operand layout (kda_fwd) */
  KDA_KERNEL_SCAN_FWD = 3,          /* the output scan (kda_fwd) */
  KDA_KERNEL_SCAN_BWD = 4,          /* reverse state-gradient scan */
  KDA_KERNEL_CHUNK_GRAD = 5,
  KDA_KERNEL_GATE_REDUCE = 6,
  KDA_KERNEL_CHUNK_LOCAL_BWD = 7,   /* backward operand layout */
  KDA_KERNEL_CHUNK_LOCAL_STATE = 8, /* state operands only (checkpoint pass) */
  KDA_KERNEL_SCAN_REC = 9,          /* forward-direction scan recording h, Vn */
  KDA_KERNEL_SCAN_STATE = 10,       /* forward-direction scan, states only */
  /* the operators around the chunked one; their units are (token, head)
     rows, tokens, or (convolution) sequences or tokens */
  KDA_KERNEL_RECURRENT = 11,
  KDA_KERNEL_GATED_NORM = 12,
  KDA_KERNEL_GATED_NORM_BWD = 13,
  KDA_KERNEL_BLOCK_NORM = 14,
  KDA_KERNEL_BLOCK_NORM_BWD = 15,
  KDA_KERNEL_SHORT_CONV = 16,
  KDA_KERNEL_SHORT_CONV_BWD = 17,
  KDA_KERNEL_SHORT_CONV_UPDATE = 18,
  KDA_KERNEL_PARAM_REDUCE = 19,     /* sums of per-block parameter gradients */
  KDA_KERNEL_COUNT = 20
};
int kda_profile_begin(void);
int kda_profile_end(int32_t *launches, double *total_ms, int64_t *units, int n);
const char *kda_kernel_name(int kind);

/* Human-readable text for a status code, including the HIP error of the
   last failed launch on this thread for KDA_ERR_HIP. */
const char *kda_status_string(int status);

#ifdef __cplusplus
}
#endif
#endif /* KDA_H */
