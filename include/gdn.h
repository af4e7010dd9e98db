/*
 * gdn.h -- C ABI of the GB300 (sm_103a) Gated DeltaNet token-mixer library.
 *
 * The mixer runs from the concatenated QKV / z / a / b projection outputs of
 * a Qwen3.5-style linear-attention layer to its gated output (the projections
 * themselves are not part of this library).  Sources, by page title and
 * section:
 *   [QDA]  "Qwen3.5 Dense Model Architecture", section "Linear Attention"
 *          (the forward listing) and section "Cache" (conv / recurrent state
 *          shapes).
 *   [RFC]  "Qwen3.5 Simulation Support Design Document", section 2.2 (the
 *          decomposed linear-attention ops), 2.4 (conv body vs conv-state
 *          update), 3.1.3 (state memory), Appendix B (chunk size 64).
 *
 * Conventions shared by every call
 * --------------------------------
 *  - All tensors are device pointers to contiguous, token-major arrays.
 *    Packed sequences are stored back to back; `cu_seqlens` (device, int32,
 *    [num_seqs + 1], cu_seqlens[0] = 0, non-decreasing, last = total_tokens)
 *    gives their bounds.  When `cu_seqlens` is NULL the tokens split into
 *    num_seqs equal sequences of total_tokens / num_seqs.
 *  - The caller owns every buffer.  The library never allocates, never frees
 *    and never synchronises: each call enqueues kernels on `stream` (a
 *    cudaStream_t passed as void*, NULL = legacy default stream) and returns.
 *  - Element types are chosen per argument with gdn_dtype.  Gates (g, beta),
 *    A_log, dt_bias, norm weights and recurrent states are always float32.
 *  - Every pointer must be 16-byte aligned.
 *  - Return value: GDN_OK, or an error code with nothing enqueued.  Argument
 *    errors are detected on the host before any launch.  A launch failure
 *    returns GDN_ERR_CUDA; gdn_last_error_string() describes the last error
 *    of the calling thread.  Inconsistent device-side metadata (a cu_seqlens
 *    that is not monotone or does not end at total_tokens; see gdn_paged_cache
 *    for the cache's) is detected on the device: the offending kernel skips the
 *    bad sequence and raises a sticky device error flag, read (and cleared) by
 *    gdn_check_device_error().
 *  - On its first use on a device the library looks up (once, with that device
 *    current) the device addresses of its own module variables: the error
 *    flag and the scratch array of gdn_chunk_prefill_static.  Those addresses
 *    belong to the device's primary context, so resetting the device
 *    (cudaDeviceReset) or destroying its primary context after the first call
 *    is not supported: later calls would use stale addresses.
 *
 * Supported sizes of the mixer: Dk, Dv in {64, 128}; Nv a multiple of Nk; conv
 * kernel 4; chunk 64.  Other sizes return GDN_ERR_UNSUPPORTED.
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GDN_OK = 0,
  GDN_ERR_INVALID_ARG = 1,  /* bad pointer, size, alignment or dtype        */
  GDN_ERR_UNSUPPORTED = 2,  /* a head size without a compiled kernel        */
  GDN_ERR_CUDA = 3,         /* a CUDA runtime error while enqueueing         */
  GDN_ERR_DEVICE = 4        /* the device error flag was raised (see above) */
} gdn_status;

typedef enum {
  GDN_BF16 = 0,  /* bfloat16 */
  GDN_F32 = 1    /* float32  */
} gdn_dtype;

/* Problem sizes shared by the calls.
 *   num_seqs      N, number of packed sequences (>= 1)
 *   total_tokens  tokens over all sequences (>= 0)
 *   num_k_heads   Nk, query/key heads;   head_k_dim Dk
 *   num_v_heads   Nv, value heads;       head_v_dim Dv
 * The concatenated projection has C = 2*Nk*Dk + Nv*Dv channels, ordered
 * [q heads | k heads | v heads] ([QDA] split of mixed_qkv).  Value head h
 * reads key head h / (Nv / Nk) (repeat_interleave of the key heads, [QDA]). */
typedef struct {
  int32_t num_seqs;
  int32_t total_tokens;
  int32_t num_k_heads;
  int32_t num_v_heads;
  int32_t head_k_dim;
  int32_t head_v_dim;
} gdn_dims;

/* Library version, (major << 16) | minor. */
int gdn_version(void);

/* Description of the last error returned on the calling thread. */
const char* gdn_last_error_string(void);

/* Synchronises `stream`, then reads and clears the device error flag.
 * Returns GDN_OK, GDN_ERR_DEVICE (flag was set) or GDN_ERR_CUDA. */
int gdn_check_device_error(void* stream);

/* ------------------------------------------------------------------------
 * gdn_conv_gating -- steps a1 + a2 + a3 of a prefill ([QDA] forward listing:
 * causal conv with cached left context, SiLU, split into heads, beta, g, and
 * the q/k L2-norm of [RFC] 2.2 op 3).
 *
 * Per sequence, with xpad = [conv_state_in (K-1 = 3 oldest-first inputs, or
 * zeros) ; x] along time and K = 4:
 *   y[t, c]  = silu( sum_j conv_w[c, j] * xpad[t + j, c] + conv_bias[c] )
 *   q[t, i]  = q_scale * y_q / sqrt(sum(y_q^2) + l2_eps)   per key head i
 *   k[t, i]  =           y_k / sqrt(sum(y_k^2) + l2_eps)   per key head i
 *   v[t, h]  = y_v                                          per value head h
 *   beta     = sigmoid(b);  g = -exp(A_log) * softplus(a + dt_bias)  (fp32)
 * On the tiled bf16 path (see the launches below) with bf16 outputs, silu(x) is
 * evaluated as h + h tanh(h), h = x / 2, with the hardware tanh: its absolute
 * error is at most about 2^-11 |h|, within half a bf16 ulp of the result for
 * x >= -2 (for more negative x the result is near zero and its relative error
 * grows); otherwise silu(x) = x / (1 + e^-x).
 *   conv_state_out[s] = the last 3 entries of xpad (raw inputs, oldest first)
 *
 *   mixed_qkv      [tokens, C]          in_dtype
 *   conv_w         [C, 4]               in_dtype (w[c,3] multiplies token t)
 *   conv_bias      [C] in_dtype, or NULL
 *   conv_state_in  [N, C, 3] in_dtype, or NULL (zero left context)
 *   conv_state_out [N, C, 3] in_dtype, or NULL (not written); may equal
 *                  conv_state_in for an in-place update
 *   a, b           [tokens, Nv]         in_dtype
 *   A_log, dt_bias [Nv]                 float32
 *   q, k           [tokens, Nk, Dk]     out_dtype
 *   v              [tokens, Nv, Dv]     out_dtype
 *   g, beta        [tokens, Nv]         float32
 * One kernel is enqueued for the conv/norm/gating pass.  A second one, the
 * conv-state update, follows when conv_state_out is not NULL and either
 * conv_state_in is not NULL (it reads the old state first, so the update may
 * be in place) or the inputs do not take the tiled bf16 path (C a multiple of
 * 1024, Nk*Dk a multiple of 256); otherwise the first kernel writes the new
 * state from its staged input rows.
 * ------------------------------------------------------------------------ */
int gdn_conv_gating(const gdn_dims* dims, const int32_t* cu_seqlens,
                    const void* mixed_qkv, int in_dtype,
                    const void* conv_w, const void* conv_bias,
                    const void* conv_state_in, void* conv_state_out,
                    const void* a, const void* b,
                    const float* A_log, const float* dt_bias,
                    float q_scale, float l2_eps,
                    void* q, void* k, void* v, int out_dtype,
                    float* g, float* beta, void* stream);

/* ------------------------------------------------------------------------
 * gdn_conv_state_steps -- the conv state after every token: the rollback
 * points of a multi-token (draft + verify) decode step, beside the recurrent
 * states of gdn_recurrent_decode_steps; a caller that accepts the first j + 1
 * tokens of a sequence keeps step_states[bos + j] as its conv state.  With
 * xpad = [conv_state_in (3 oldest-first inputs, or zeros) ; x] of a sequence
 * ([QDA] "Cache": the conv cache keeps the latest raw inputs), token i of it
 * gets step_states[bos + i] = xpad[i + 1 .. i + 3] (oldest first).  The last
 * token's entry equals the conv_state_out of gdn_conv_gating.
 *   mixed_qkv      [tokens, C]          in_dtype
 *   conv_state_in  [N, C, 3] in_dtype, or NULL (zeros); the state the tokens
 *                  follow -- read it before an in-place update of it
 *   step_states    [tokens, C, 3]       in_dtype, written
 * ------------------------------------------------------------------------ */
int gdn_conv_state_steps(const gdn_dims* dims, const int32_t* cu_seqlens, const void* mixed_qkv, int in_dtype,
                         const void* conv_state_in, void* step_states, void* stream);

/* ------------------------------------------------------------------------
 * gdn_gating -- step a3 alone, for callers that already hold q, k, v:
 *   beta[t, h] = sigmoid(b[t, h]);  g[t, h] = -exp(A_log[h]) * softplus(a[t, h] + dt_bias[h])
 *   a, b [rows, Nv] in_dtype; A_log, dt_bias [Nv] float32; g, beta [rows, Nv] float32.
 * ([QDA] forward listing: beta = b.sigmoid(), g in float32.)
 * ------------------------------------------------------------------------ */
int gdn_gating(int64_t rows, int32_t num_v_heads, const void* a, const void* b, int in_dtype,
               const float* A_log, const float* dt_bias, float* g, float* beta, void* stream);

/* ------------------------------------------------------------------------
 * gdn_chunk_prefill -- step a4: the chunked gated delta rule ([RFC] 2.2 op 4,
 * Appendix B: chunk 64, intra-chunk attention + inter-chunk recurrence;
 * [QDA] chunk_gated_delta_rule with initial_state / output_final_state).
 *
 * Computes exactly the recurrence of gdn_recurrent_decode over every token of
 * every sequence, chunk by chunk (chunks restart at each sequence start):
 *   S <- exp(g_t) S;  u = beta_t (v_t - S^T k_t);  S <- S + k_t u^T;
 *   o_t = S^T (scale * q_t),     S in [Dk, Dv] layout, fp32.
 * bf16 q, k, v with Dk = Dv = 128 run on the tensor cores (bf16 products,
 * fp32 accumulation and state); fp32 inputs and 64-wide heads run the fp32
 * CUDA-core kernel of gdn_chunk_prefill_fp32.
 *
 * Launches: on the tensor-core path, a memset of the workspace's flags and
 * then, for one sequence, a single cooperative launch (one CTA per SM; the
 * scan of each head overlaps the solve of later chunks), or, for packed
 * batches, a solve kernel and a scan kernel.  One long sequence (32 chunks or
 * more) runs split in two segments when the device holds three scans per head
 * and two solve CTAs per head beside them (with Nv = 32 that needs 160 SMs):
 * the second segment is scanned from a zero state and its transition map beside
 * the first, and a fix-up kernel adds the first segment's final state's share
 * to its outputs and to the final state.
 * The workspace of one sequence holds a ring of 16 solve-tile positions per
 * head (and segment), one flag per (chunk, head), and the split's scratch when
 * it splits: it grows by 4 bytes per chunk and head (plus, split, 128 bytes per
 * token and head), not by the 49,664-byte tile of every chunk.  Packed batches
 * keep one tile per (chunk, head).  The size is for the current device (its SM
 * count decides the split).  One workspace must not be shared by calls that
 * can run at the same time.
 *
 *   q, k           [tokens, Nk, Dk]     in_dtype
 *   v              [tokens, Nv, Dv]     in_dtype
 *   g, beta        [tokens, Nv]         float32
 *   scale          multiplies q (1.0 when q comes from gdn_conv_gating)
 *   initial_state  [N, Nv, Dk, Dv] float32, or NULL (zero state)
 *   final_state    [N, Nv, Dk, Dv] float32, or NULL (not written); may
 *                  equal initial_state (in-place update)
 *   o              [tokens, Nv, Dv]     out_dtype
 *   workspace      device scratch of gdn_chunk_prefill_workspace_size()
 *                  bytes (may be NULL when that size is 0)
 * ------------------------------------------------------------------------ */
int gdn_chunk_prefill_workspace_size(const gdn_dims* dims, size_t* bytes);

int gdn_chunk_prefill(const gdn_dims* dims, const int32_t* cu_seqlens,
                      const void* q, const void* k, const void* v, int in_dtype,
                      const float* g, const float* beta, float scale,
                      const float* initial_state, float* final_state,
                      void* o, int out_dtype,
                      void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * gdn_chunk_prefill_gated_norm -- steps a4 + a6 in one pass: the chunked
 * gated delta rule of gdn_chunk_prefill followed by the gated RMSNorm of
 * gdn_gated_rmsnorm on each (token, value head) row of its output
 * ([RFC] 2.2 ops 4 and 6; [QDA] forward listing: core output, then
 * self.norm(core_output, z)).  The core output o is rounded to bf16 (as a
 * stored bf16 o would be) and normalised:
 *   y[t, h] = o[t, h] / sqrt(mean(o[t, h]^2) + norm_eps) * norm_w * silu(z[t, h])
 * One sequence (the cooperative launch): the scan stores o into y and spare
 * solve groups normalise each 64-token block in place once it has landed, beside
 * the scan of later chunks (on one GB300, 119.2 us against 111.1 + 18.9 us for
 * gdn_chunk_prefill + gdn_gated_rmsnorm at 4096 tokens, 32 heads).  Packed
 * batches apply the norm in the scan's output epilogue (o is never stored; for
 * bf16 y the gate norm_w * silu(z) is evaluated in bf16x2 arithmetic), which is
 * slower than the two separate calls.  fp32 y keeps fp32 arithmetic.
 * Arguments as gdn_chunk_prefill, with o replaced by
 *   z              [tokens, Nv, Dv]     bf16 (else GDN_ERR_UNSUPPORTED)
 *   norm_w         [Dv]                 float32
 *   norm_eps       the RMSNorm epsilon
 *   y              [tokens, Nv, Dv]     out_dtype
 * Tensor-core shapes only (bf16 q/k/v, Dk = Dv = 128; else
 * GDN_ERR_UNSUPPORTED); same workspace as gdn_chunk_prefill.
 * ------------------------------------------------------------------------ */
int gdn_chunk_prefill_gated_norm(const gdn_dims* dims, const int32_t* cu_seqlens,
                                 const void* q, const void* k, const void* v, int in_dtype,
                                 const float* g, const float* beta, float scale,
                                 const float* initial_state, float* final_state,
                                 const void* z, int z_dtype, const float* norm_w, float norm_eps,
                                 void* y, int out_dtype,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* gdn_chunk_prefill_fp32 -- the same computation as gdn_chunk_prefill, on
 * CUDA cores in fp32 throughout (q, k, v are not rounded to bf16).  Slower;
 * for callers that want fp32 accuracy of the chunk form.  Same arguments,
 * no workspace. */
int gdn_chunk_prefill_fp32(const gdn_dims* dims, const int32_t* cu_seqlens,
                           const void* q, const void* k, const void* v, int in_dtype,
                           const float* g, const float* beta, float scale,
                           const float* initial_state, float* final_state,
                           void* o, int out_dtype, void* stream);

/* gdn_chunk_prefill_static -- gdn_chunk_prefill for callers that cannot
 * allocate device memory: hosts that reserve the device's memory up front
 * (a serving engine's arena, another framework's plugin interface) and have
 * no allocator to hand out a workspace at call time.  No counterpart on the
 * source pages; this is a packaging choice of the library.
 *
 * Same arguments as gdn_chunk_prefill without the workspace: the library uses
 * its own fixed 32 MiB scratch array in device memory instead, which every
 * GPU that loads the library holds until the process exits.  This call never
 * allocates or frees.
 *   - Supported inputs: bf16 q/k/v with Dk = Dv = 128 (else
 *     GDN_ERR_UNSUPPORTED).
 *   - Size limit: the workspace of these dims, laid out without the split of a
 *     long sequence, must be at most 32 MiB.  One sequence of any length up to
 *     about 2 million tokens fits (its solve tiles go through a fixed ring; at
 *     32 value heads the ring takes 25.4 MB), but it never runs split.  Packed
 *     batches keep a tile per (chunk, head): at 32 value heads, about 1,200
 *     tokens in all.  Larger problems return GDN_ERR_INVALID_ARG and should use
 *     gdn_chunk_prefill.
 *   - The first call on a device looks up the scratch array's device address
 *     (once per device, with that device current); make that first call before
 *     any stream capture.
 *   - All calls share the one array and it keeps the last call's contents
 *     (every call rewrites what it reads, so nothing needs clearing).  Calls
 *     that overlap on the GPU (different streams, or different host threads)
 *     race on it: serialise them. */
int gdn_chunk_prefill_static(const gdn_dims* dims, const int32_t* cu_seqlens,
                             const void* q, const void* k, const void* v, int in_dtype,
                             const float* g, const float* beta, float scale,
                             const float* initial_state, float* final_state,
                             void* o, int out_dtype, void* stream);

/* ------------------------------------------------------------------------
 * gdn_recurrent_decode -- step a5: the token-by-token gated delta rule with
 * the fp32 state read-modify-written in place ([RFC] 2.2 op 5 and 3.1.3
 * state memory; [QDA] recurrent_gated_delta_rule).  For every sequence and
 * value head h (key head h / (Nv/Nk)), for each of its tokens in order:
 *   S <- exp(g_t) S;  u = beta_t (v_t - S^T k_t);  S <- S + k_t u^T;
 *   o_t = S^T (scale * q_t).
 *   q, k [tokens, Nk, Dk], v [tokens, Nv, Dv]   in_dtype
 *   g, beta [tokens, Nv] float32
 *   state  [N, Nv, Dk, Dv] float32, read and overwritten in place
 *   o      [tokens, Nv, Dv] out_dtype
 * Sequences may hold several tokens (multi-token decode / verify).
 * ------------------------------------------------------------------------ */
int gdn_recurrent_decode(const gdn_dims* dims, const int32_t* cu_seqlens,
                         const void* q, const void* k, const void* v, int in_dtype,
                         const float* g, const float* beta, float scale,
                         float* state, void* o, int out_dtype, void* stream);

/* ------------------------------------------------------------------------
 * gdn_recurrent_decode_steps -- gdn_recurrent_decode that also writes the
 * state after every token: the rollback points of a multi-token (draft +
 * verify) decode step, where a caller keeps the state after the last
 * accepted token by copying step_states[bos + j] into state.  No counterpart
 * on the source pages beyond the multi-token decode itself ([QDA]
 * recurrent_gated_delta_rule over several tokens).
 *   step_states    [tokens, Nv, Dk, Dv] float32, written: the state after
 *                  token t of its sequence (same [Dk, Dv] layout as state);
 *                  NULL returns GDN_ERR_INVALID_ARG
 * Other arguments and the in-place final state as gdn_recurrent_decode.
 * ------------------------------------------------------------------------ */
int gdn_recurrent_decode_steps(const gdn_dims* dims, const int32_t* cu_seqlens,
                               const void* q, const void* k, const void* v, int in_dtype,
                               const float* g, const float* beta, float scale,
                               float* state, float* step_states, void* o, int out_dtype,
                               void* stream);

/* ------------------------------------------------------------------------
 * gdn_gated_rmsnorm -- step a6 ([RFC] 2.2 op 6, [QDA] self.norm(core, z)):
 *   y[r, :] = x[r, :] / sqrt(mean(x[r, :]^2) + eps) * w * silu(z[r, :])
 *   x [rows, dim] x_dtype; z [rows, dim] z_dtype; w [dim] float32;
 *   y [rows, dim] out_dtype.  dim in {64, 128}.
 * silu(z) as in gdn_conv_gating: the hardware-tanh form for bf16 y (absolute
 * error at most about 2^-11 |z| / 2), z / (1 + e^-z) for fp32 y.
 * ------------------------------------------------------------------------ */
int gdn_gated_rmsnorm(int64_t rows, int32_t dim, const void* x, int x_dtype,
                      const void* z, int z_dtype, const float* w, float eps,
                      void* y, int out_dtype, void* stream);

/* ------------------------------------------------------------------------
 * gdn_decode_fused -- step a7: one decode step of the whole mixer for
 * num_seqs sequences with one new token each (total_tokens == num_seqs),
 * in one launch: conv-state update + conv + SiLU ([RFC] 2.4 conv-state
 * update), split / L2-norm / q scale, gating, one recurrent step with the
 * fp32 state updated in place, and the gated RMSNorm.
 *   mixed_qkv  [B, C] in_dtype;  conv_w [C, 4] in_dtype;  conv_bias [C] or NULL
 *   conv_state [B, C, 3] in_dtype, updated in place
 *   a, b [B, Nv] in_dtype;  A_log, dt_bias [Nv] float32
 *   state [B, Nv, Dk, Dv] float32, updated in place
 *   z [B, Nv, Dv] in_dtype;  norm_w [Dv] float32
 *   y [B, Nv, Dv] out_dtype
 * ------------------------------------------------------------------------ */
int gdn_decode_fused(const gdn_dims* dims,
                     const void* mixed_qkv, int in_dtype,
                     const void* conv_w, const void* conv_bias, void* conv_state,
                     const void* a, const void* b,
                     const float* A_log, const float* dt_bias,
                     float q_scale, float l2_eps,
                     float* state, const void* z, const float* norm_w, float norm_eps,
                     void* y, int out_dtype, void* stream);

/* ------------------------------------------------------------------------
 * Softmax attention over a paged cache: the serving calls for the
 * full-attention layers that a hybrid decoder interleaves with the mixer
 * ([QDA], the full-attention layers: RMSNorm of q and k per head, partial
 * rotation, grouped query heads, sigmoid output gate; section "Cache": keys and
 * values kept per position).  Query head h reads key/value head h / (Nq / Nkv).
 *
 *   gdn_qk_norm_rope        norm + rotation of q and k, dense outputs
 *   gdn_paged_kv_append     norm + rotation of q and k, k and v into the cache
 *   gdn_paged_attn_decode   attention of the new tokens over the cache
 *
 * Head sizes 64, 128 and 256 (else GDN_ERR_UNSUPPORTED).
 * ------------------------------------------------------------------------ */

/* Sizes: N sequences, total_tokens new tokens over all of them (bounds from
 * cu_seqlens as above), Nq query heads, a multiple of Nkv, head size D. */
typedef struct {
  int32_t num_seqs;
  int32_t total_tokens;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
} gdn_attn_dims;

/* An input [tokens, heads, D] whose head rows are contiguous: element
 * (t, h, i) is data[t * token_stride + h * head_stride + i].  Strides are in
 * elements, >= 0 and multiples of 16 bytes, so that q, k, v or a gate can be a
 * slice of a joint projection output. */
typedef struct {
  const void* data;
  int64_t token_stride;
  int64_t head_stride;
} gdn_heads;

/* Per-head RMSNorm and rotation of q and k, computed in float32 and rounded
 * once when stored.
 *   q_norm_w, k_norm_w  [D] float32, or NULL (that one is not normalised):
 *                       u = x / sqrt(mean(x^2) + norm_eps) * w
 *                       (a layer that defines its weight as 1 + w passes 1 + w)
 *   cos_sin             [max_positions, rotary_dim] float32: row p holds the
 *                       rotary_dim / 2 cosines of position p, then its sines
 *                       (made by the caller, in float64 for far positions);
 *                       NULL when rotary_dim = 0 (no rotation)
 *   rotary_dim          r: the first r elements of a head are rotated, the
 *                       others pass; a multiple of 16, at most D
 *   interleaved         0: element i is paired with i + r/2;  1: 2i with 2i+1
 *                       (a, b) -> (a cos_i - b sin_i, b cos_i + a sin_i)
 *   positions           [tokens] int32 table rows, or NULL: the token's index
 *                       in its sequence (gdn_qk_norm_rope) or its index in the
 *                       cache (gdn_paged_kv_append)
 * A position outside [0, max_positions) raises the device error flag, and
 * nothing is written for its token. */
typedef struct {
  const float* q_norm_w;
  const float* k_norm_w;
  float norm_eps;
  int32_t rotary_dim;
  int32_t interleaved;
  int32_t max_positions;
  const float* cos_sin;
  const int32_t* positions;
} gdn_norm_rope;

/* A paged key/value cache.  Element i of slot j of key/value head h in page p
 * is at p * page_stride + h * head_stride + j * slot_stride + i of k and of v
 * (strides in elements, positive multiples of 16 bytes, below 2^40 bytes), so
 * both a [pages, Nkv, page_size, D] and a [pages, page_size, Nkv, D] cache, or
 * the two halves of a [pages, 2, ...] one, can be passed.  In order of size,
 * the strides of the axes with more than one entry are at least D and what the
 * axis below spans (no two entries overlap), and each is a multiple of the one
 * below (else GDN_ERR_UNSUPPORTED).
 *   block_table  [N, max_pages] int32: index p of sequence s lives in slot
 *                p % page_size of page block_table[s, p / page_size]; entries
 *                past a sequence's length are not read
 *   kv_lens      [N] int32: the sequence's cached tokens INCLUDING the call's
 *                new ones: new token i of n has cache index kv_lens[s] - n + i.
 *                0 marks an inactive slot of a padded batch.
 * A length below 0, below the sequence's new tokens (unless 0) or above
 * max_pages * page_size (the attention's limit is also 2^31 - 256), and a page
 * id outside [0, num_pages), raise the device error flag. */
typedef struct {
  void* k;
  void* v;
  int64_t page_stride;
  int64_t head_stride;
  int64_t slot_stride;
  int32_t num_pages;
  int32_t page_size;
  int32_t max_pages;
  const int32_t* block_table;
  const int32_t* kv_lens;
} gdn_paged_cache;

/* ------------------------------------------------------------------------
 * gdn_qk_norm_rope -- per-head norm and rotation of queries and keys.
 *   q [tokens, Nq, D], k [tokens, Nkv, D]   in_dtype (strided, see gdn_heads);
 *                                           k may be NULL (q alone)
 *   q_out [tokens, Nq, D], k_out [tokens, Nkv, D]   out_dtype, contiguous;
 *       may be the input's own memory when that is contiguous and of the same
 *       type, and must not overlap an input otherwise
 * ------------------------------------------------------------------------ */
int gdn_qk_norm_rope(const gdn_attn_dims* dims, const int32_t* cu_seqlens,
                     const gdn_heads* q, const gdn_heads* k, int in_dtype,
                     const gdn_norm_rope* nr,
                     void* q_out, void* k_out, int out_dtype, void* stream);

/* ------------------------------------------------------------------------
 * gdn_paged_kv_append -- writes the new tokens' keys (normed and rotated on
 * the way) and values into the cache, and norms and rotates q beside them.
 *   q              NULL: only k and v;  else q_out [tokens, Nq, D] q_dtype,
 *                  contiguous (may be q's own memory, as above)
 *   k, v           [tokens, Nkv, D]   in_dtype (strided)
 *   nr             NULL: neither norm nor rotation
 *   cache          written in cache_dtype; read: block_table and kv_lens
 * Nothing is written for an inactive sequence (kv_lens = 0; q_out neither) nor
 * for a token whose metadata raised the error flag.  Two tokens that map to
 * one slot leave a mix of their rows there, in pieces of 16 bytes.
 * ------------------------------------------------------------------------ */
int gdn_paged_kv_append(const gdn_attn_dims* dims, const int32_t* cu_seqlens,
                        const gdn_heads* q, const gdn_heads* k, const gdn_heads* v,
                        int in_dtype, const gdn_norm_rope* nr,
                        const gdn_paged_cache* cache, int cache_dtype,
                        void* q_out, int q_dtype, void* stream);

/* ------------------------------------------------------------------------
 * gdn_paged_attn_decode -- attention of the new tokens of each sequence over
 * its cache (whose last entries are the new tokens' own, appended before):
 *   o[t, h] = sum_j softmax_j(scale * q[t, h] . k_j) v_j   over the cache
 *             indices j up to the token's own
 *   y[t, h] = o[t, h] * sigmoid(gate[t, h])                when gate is given
 * Rows of an inactive sequence (kv_lens = 0) and of one whose kv_lens raised
 * the error flag are zero; a page id that raised it reads as zeros.  Cache
 * entries past a token's own index never reach its row, whatever they hold.
 * Scores, softmax statistics and sums are float32.  With a bf16 cache the
 * weights enter the product with v as the sum of two bf16 values, 16 bits of
 * them (2^-16 relative to sum_j p_j |v_j|: below the rounding of a bf16 o, to be
 * seen in a float32 one).  A visible NaN, or an infinite v, makes what it
 * enters NaN or infinite (with a bf16 cache NaN also where an infinite v alone
 * would give infinity).
 *
 * Made for one or a few new tokens per sequence (decode, draft + verify): up
 * to 8 query heads of one token and one key/value head are one tile of the
 * products (float32: up to 4 or 8), a few tiles share one pass over the
 * sequence's whole cache, and a sequence with more tokens takes more passes.
 *
 *   q, gate    [tokens, Nq, D]   in_dtype (strided); gate may be NULL
 *   cache      in_dtype
 *   o          [tokens, Nq, D]   out_dtype, contiguous
 *   workspace  device scratch of gdn_paged_attn_decode_workspace_size() bytes
 *              (may be NULL when that is 0), no initialisation needed; not to
 *              be shared by calls that can run at the same time.  The size is
 *              for the current device and for tables of up to table_tokens =
 *              max_pages * page_size cache entries: it is 0 for short tables
 *              and the same for all others, and depends on the heads, D and the
 *              type, not on the numbers of sequences and tokens (20 MB at most
 *              on 152 SMs; one token may use as little as a quarter of it).
 * ------------------------------------------------------------------------ */
int gdn_paged_attn_decode_workspace_size(const gdn_attn_dims* dims, int in_dtype, int64_t table_tokens,
                                         size_t* bytes);

int gdn_paged_attn_decode(const gdn_attn_dims* dims, const int32_t* cu_seqlens,
                          const gdn_heads* q, const gdn_heads* gate, int in_dtype,
                          const gdn_paged_cache* cache, float scale,
                          void* o, int out_dtype,
                          void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * The same cache in 4 bits, for head sizes 64, 128 and 256: 4.5 bits an element
 * instead of 16.  No counterpart on the source pages beyond the cache itself.
 * A head row is held in groups of 64 elements.  Of a group x (after norm and
 * rotation) with least value lo and greatest hi the cache holds
 *   m = bf16(lo),  s = bf16((hi - lo) / 15),  n_i = round((x_i - m) / s) in 0 .. 15
 * (halves to even; lo and (hi - lo) / 15 are rounded to float32 first), and element i
 * reads as n_i s + m.  Roundings are decided as from float64 values: what is stored
 * does not depend on the order of any sum.  A group of one value (and
 * one whose step would be below 2^-100) has s = 0, n = 0; one that holds an
 * infinity or NaN, or whose range passes float32, reads as NaN.
 *
 *   gdn_paged_kv4_append       norm + rotation of q and k, k and v into the cache
 *   gdn_paged_kv4_read         cached tokens as dense keys and values
 *   gdn_paged_kv4_attn_decode  attention of the new tokens over the cache
 *
 * k, v            bytes: element 2 i of slot j of head h in page p is the low half,
 *                 2 i + 1 the high half, of byte p * page_stride + h * head_stride
 *                 + j * slot_stride + i  (strides in bytes, positive multiples of
 *                 16, below 2^36)
 * k_scale, v_scale   bf16 pairs (s, m): group g at element p * scale_page_stride +
 *                 h * scale_head_stride + j * scale_slot_stride + 2 g (strides in
 *                 bf16 elements, positive multiples of the row's D / 32, below 2^33)
 * No two rows overlap (else GDN_ERR_INVALID_ARG).  The other fields as in
 * gdn_paged_cache. */
typedef struct {
  void* k;
  void* v;
  void* k_scale;
  void* v_scale;
  int64_t page_stride;
  int64_t head_stride;
  int64_t slot_stride;
  int64_t scale_page_stride;
  int64_t scale_head_stride;
  int64_t scale_slot_stride;
  int32_t num_pages;
  int32_t page_size;
  int32_t max_pages;
  const int32_t* block_table;
  const int32_t* kv_lens;
} gdn_paged_cache4;

/* gdn_paged_kv4_append -- gdn_paged_kv_append into a 4-bit cache: the same
 * arguments, and the same rules for inactive sequences and bad metadata.  Two
 * tokens that map to one slot leave a mix of their rows there, in pieces of 4
 * bytes, under either's scales. */
int gdn_paged_kv4_append(const gdn_attn_dims* dims, const int32_t* cu_seqlens,
                         const gdn_heads* q, const gdn_heads* k, const gdn_heads* v,
                         int in_dtype, const gdn_norm_rope* nr,
                         const gdn_paged_cache4* cache, void* q_out, int q_dtype, void* stream);

/* ------------------------------------------------------------------------
 * gdn_paged_kv4_read -- the values that the cache holds, dense: for what does not
 * read 4 bits itself (the attention of a prompt's next part over its cached
 * part, a copy of a cache).  Row i of the n rows of a sequence (bounds from
 * cu_seqlens, as for the other calls) is its cache index kv_lens[s] - n + i: with
 * n = kv_lens[s] the whole sequence.
 *   k_out, v_out   [tokens, Nkv, D] out_dtype, contiguous; one may be NULL
 * Rows of an inactive sequence (kv_lens = 0), and of metadata that raised the
 * error flag, are zero.  dims->num_q_heads is not used (a multiple of Nkv).
 * ------------------------------------------------------------------------ */
int gdn_paged_kv4_read(const gdn_attn_dims* dims, const int32_t* cu_seqlens,
                       const gdn_paged_cache4* cache, void* k_out, void* v_out, int out_dtype,
                       void* stream);

/* ------------------------------------------------------------------------
 * gdn_paged_kv4_attn_decode -- gdn_paged_attn_decode over a 4-bit cache: the same
 * formulas, and the same rules for inactive sequences, bad metadata and entries
 * past a token's own index.  Scores, softmax statistics and sums are float32; a
 * weight times a step enters the product with the numbers n in f16 (2^-11 relative to
 * sum_j p_j s_j n_j: an eighth of the rounding of a bf16 output; one below 2^-17 of the
 * row's largest p_j s_j in the group is off by up to 2^-27 of that), and a query's elements
 * too, next to a power of two of the row's own (off by up to 2^-31 of its largest).  A row's
 * bits may differ with the other sequences of the call (the order of its sums does).
 *   q, gate    [tokens, Nq, D]   bf16 (strided); gate may be NULL
 *   o          [tokens, Nq, D]   bf16, contiguous
 *   workspace  device scratch of gdn_paged_kv4_attn_decode_workspace_size() bytes
 *              (may be NULL when that is 0), no initialisation needed; not to be
 *              shared by calls that can run at the same time.  For the current device
 *              and tables of up to table_tokens = max_pages * page_size entries: 0
 *              for short tables, else the same for all numbers of sequences and tokens
 *              (5.2 MB at most on 152 SMs).
 * total_tokens * num_q_heads is below 2^31 (else GDN_ERR_UNSUPPORTED).
 * ------------------------------------------------------------------------ */
int gdn_paged_kv4_attn_decode_workspace_size(const gdn_attn_dims* dims, int64_t table_tokens, size_t* bytes);

int gdn_paged_kv4_attn_decode(const gdn_attn_dims* dims, const int32_t* cu_seqlens,
                              const gdn_heads* q, const gdn_heads* gate,
                              const gdn_paged_cache4* cache, float scale, void* o,
                              void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * gdn_paged_plan -- the paged cache's metadata of the next step, from the lengths
 * of its requests: pages from a ring of free ones into the block table, the
 * bounds of the packed new tokens, their positions and cache slots.  One launch,
 * nothing read on the host: a captured step follows its requests.
 *
 *   new_lens    [N]  the step's new tokens of each sequence; 0: none, it stays as
 *                    it is; < 0: it has ended, its pages go back; GDN_PLAN_REST, of the
 *                    last sequence alone (with kv_lens 0): the rows up to total_tokens
 *                    that the others leave, as those of an inactive slot (kv_lens_out
 *                    0, no pages), which makes a step of any tokens one of total_tokens
 *   kv_lens     [N]  cached tokens before the step (gdn_draft_verify's kv_lens_out
 *                    after refused drafts)
 *   pages_held  [N]  pages of the sequence, the first so many of its table row; may
 *                    be more than its tokens need
 *   free_ring   [2]  h, c: the c free pages are free_pages[(h + i) % num_pages].  Every
 *                    page is free or held by one sequence (none shares a prefix)
 * Sequence after sequence takes what it lacks, max(0, ceil((kv_lens + new_lens) /
 * page_size) - pages_held) pages, from the front of the ring; pages of ended
 * sequences go behind its end (and are given out by a later call).
 *   block_table [N, max_pages], free_pages [num_pages]   updated in place
 *   cu_seqlens  [N + 1]         prefix sums of max(new_lens, 0)
 *   positions   [total_tokens]  each new token's cache index, or NULL
 *   slots       [total_tokens]  its page * page_size + slot, or NULL (for calls of the
 *                               user's own; this library's go by the block table)
 *   kv_lens_out, pages_held_out, free_ring_out   the state after the step; each may
 *                               be its input.  Ended sequences have length 0.
 * total_tokens rows that the new tokens do not fill have position 0 and slot -1
 * (the other calls want cu_seqlens to end at their total_tokens: GDN_PLAN_REST).
 *
 * All or nothing: where pages run out, a table row or total_tokens is too short,
 * or the state is inconsistent (kv_lens above pages_held * page_size, below 0, more
 * pages free and given back than there are, ...),
 * the device error flag is raised, the state stays as it was and the step has no
 * tokens.  A page id outside [0, num_pages) that a new token needs, or that is taken or
 * given back, raises the flag; the slots of its tokens are -1, and it stays where it
 * is, in the table or in the ring.
 * At most 16384 sequences (else GDN_ERR_UNSUPPORTED).
 * ------------------------------------------------------------------------ */
#define GDN_PLAN_REST 0x7fffffff

typedef struct {
  int32_t num_seqs;
  int32_t total_tokens;
  int32_t num_pages;
  int32_t page_size;
  int32_t max_pages;
  const int32_t* new_lens;
  const int32_t* kv_lens;
  const int32_t* pages_held;
  const int32_t* free_ring;
  int32_t* free_pages;
  int32_t* block_table;
  int32_t* cu_seqlens;
  int32_t* positions;
  int64_t* slots;
  int32_t* kv_lens_out;
  int32_t* pages_held_out;
  int32_t* free_ring_out;
} gdn_page_plan;

int gdn_paged_plan(const gdn_page_plan* plan, void* stream);

/* ------------------------------------------------------------------------
 * gdn_draft_verify -- which drafted tokens of a multi-token step stay, and the
 * token behind them, so that what is kept is distributed as the target model's
 * own samples.  Beside gdn_recurrent_decode_steps and gdn_conv_state_steps, whose
 * states after row bos + accepted[s] are those to go on with.
 *
 * Sequence s has the n rows [bos, eos) of the step (cu_seqlens, or equally many):
 * tokens[bos] is certain, tokens[bos + 1 ..] are its n - 1 drafts, and row bos + i
 * of target_probs is the target's distribution behind token i.  In a step that also
 * has prompts these rows are fewer than gdn_paged_plan's: a prompt's last token alone
 * (n = 1), whose probabilities are the only ones needed, so the call gets cu_seqlens of
 * its own.  Draft x = tokens[bos
 * + i + 1] is kept while
 *   uniform[bos + i] * draft_probs[s, i, x] < target_probs[bos + i, x]   (in order)
 * with draft_probs counted as 1 at x where none are given (drafts that were looked
 * up, not drawn).  With a drafts kept the next token is drawn from the weights
 *   w = max(target_probs[bos + a] - draft_probs[s, a], 0)  if a draft was refused (no
 *       draft_probs: target_probs without the refused token; where that leaves
 *       nothing: target_probs[bos + a]),
 *   w = target_probs[bos + a]                              if all were kept,
 * by U = floor(uniform[eos - 1] * 2^24): the least j with C_j 2^24 > U W, C the
 * running sum of w and W its end.  p and q enter w in whole units of 2^-42 (halves to
 * even), so that the sums, and the result, do not depend on any order.  Probabilities
 * below 0 or NaN count as 0, above 1 as 1, in w; NaN refuses a draft.
 *   target_probs  [T, V] prob_dtype, rows target_row elements apart
 *   draft_probs   [N, max_drafts, V] prob_dtype or NULL: sequences draft_seq, rows
 *                 draft_row elements apart
 *   tokens        [T] int32;  uniform [T] float32 in [0, 1)
 *   accepted      [N] int32: a;  0 for a sequence without rows
 *   out_tokens    [T] int32, not tokens itself: rows bos .. bos + a - 1 the drafts kept, bos + a the token
 *                 drawn, the others -1
 *   kv_lens, kv_lens_out  [N] int32 or both NULL: kv_lens_out = kv_lens - (n - 1 - a),
 *                 the cached tokens that stay; may be the same.  kv_lens counts the
 *                 step's tokens (gdn_paged_plan's kv_lens_out); fewer than the refused
 *                 ones give a length below 0, which gdn_paged_plan refuses.  Length 0 marks
 *                 an inactive slot of a padded batch: a = 0, its out_tokens -1
 * A draft outside [0, V) or without a row of draft_probs is refused, and a row that
 * has no weight draws -1; both raise the device error flag.
 * V at most 2^21 (else GDN_ERR_UNSUPPORTED).
 * ------------------------------------------------------------------------ */
int gdn_draft_verify(int32_t num_seqs, int32_t total_tokens, int32_t vocab, int32_t max_drafts,
                     const int32_t* cu_seqlens,
                     const void* target_probs, int64_t target_row,
                     const void* draft_probs, int64_t draft_seq, int64_t draft_row, int prob_dtype,
                     const int32_t* tokens, const float* uniform,
                     const int32_t* kv_lens, int32_t* kv_lens_out,
                     int32_t* accepted, int32_t* out_tokens, void* stream);

/* ------------------------------------------------------------------------
 * Test hook (no counterpart on the source pages): failure detection of the
 * bounded device waits.  Every wait of the chunk-prefill scan on a ready flag
 * or an mbarrier gives up after a bound of device time (2 s in the calls
 * above); the CTA then lets its copies and products in flight land, releases
 * its tensor memory, raises the device error flag with code 2 ("bounded wait
 * timed out") and exits, and the context stays usable.
 *
 * gdn_test_chunk_wait_timeout enqueues the one-sequence chunk-prefill launch
 * of gdn_chunk_prefill with no solve work, so that no chunk's ready flag is
 * ever published, and with each wait bounded by wait_ns (1 ms .. 10 s): every
 * scan's first flag wait runs out while none of its copies or products is in
 * flight.  Arguments as gdn_chunk_prefill (one sequence, bf16 q/k/v and o,
 * Dk = Dv = 128, no states); o is not written.  The caller then reads
 * GDN_ERR_DEVICE from gdn_check_device_error().  Returns GDN_ERR_UNSUPPORTED
 * when the device cannot hold the one-sequence launch (fewer SMs than value
 * heads + 1, or no cooperative launch).
 * ------------------------------------------------------------------------ */
int gdn_test_chunk_wait_timeout(const gdn_dims* dims, const void* q, const void* k, const void* v,
                                const float* g, const float* beta, void* o, void* workspace,
                                size_t workspace_bytes, int64_t wait_ns, void* stream);

/* gdn_test_paged_attn_wait_timeout enqueues gdn_paged_attn_decode (o in
 * in_dtype, no gate, scale 1) with copies that are never issued although the
 * kernel waits for them (skip: 1 query rows, 2 keys and values, 3 both), and
 * with each wait bounded by wait_ns (1 ms .. 10 s): every CTA with work gives
 * up, lets what it has in flight land, raises the device error flag with code 2
 * and exits.  What o then holds is undefined. */
int gdn_test_paged_attn_wait_timeout(const gdn_attn_dims* dims, const int32_t* cu_seqlens,
                                     const gdn_heads* q, int in_dtype, const gdn_paged_cache* cache,
                                     void* o, void* workspace, size_t workspace_bytes,
                                     int64_t wait_ns, int skip, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H_ */
