/*
 * muon_attention.h — the attention half of a block beside the layers of
 * muon_layers.h, in the same library (libmuon_ns.so), for MI355X (gfx950):
 *
 *   muon_rotary          queries and keys turned by their positions
 *   muon_diff_attention  differential attention: the difference of two softmax
 *                        maps, one of them weighted by a learned λ
 *   muon_dropout         dropout and the residual's addition
 *
 * each with its backward pass.  Conventions are those of muon_layers.h:
 * device pointers owned by the caller, kernel launches only on `stream`,
 * every argument checked on the host before anything is enqueued, status codes
 * with muon_last_error(), MUON_DEBUG_SYNC=1, no C++ exception across the
 * boundary, 256-byte aligned caller-allocated workspaces that overlap no
 * tensor of the call, dtype MUON_DTYPE_F32 or MUON_DTYPE_BF16, fp32 sums and
 * statistics, outputs rounded once, sums in a fixed order that depends on the
 * sizes alone.  These calls add entry points only: MUON_NS_ABI_VERSION is
 * unchanged.
 *
 * Tensors of heads have the sizes batch × tokens × heads × values with the
 * values of a head contiguous and a stride for each of the other three, in
 * elements (0 … 2^40, any order: heads may lie outside tokens).  An input's
 * elements may coincide (stride 0); an output's may not.  Any alignment of the
 * element type is accepted.
 *
 * An output may not overlap an input or another output unless the entry point
 * says so (MUON_ERR_ALIAS).  Overlap is judged by address ranges, except that
 * tensors of one token stride (of one token each: batch stride) that interleave,
 * as queries and keys of one fused projection do, count as apart.
 */
#ifndef MUON_ATTENTION_H
#define MUON_ATTENTION_H

#include "muon_layers.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ----- rotary positions --------------------------------------------------- */

/* Pair i < rotated/2 of a head, values i and rotated/2 + i (interleaved = 0) or
 * 2i and 2i + 1 (interleaved = 1), turns by θ = position · freqs[i]:
 *   (a, b) → scale · (a·cosθ − b·sinθ, a·sinθ + b·cosθ);
 * the other dim − rotated values stay as they are.
 *   freqs: rotated/2 doubles, radians per position.  θ is formed and reduced in
 *     fp64, so far positions lose nothing.
 *   positions: int32 or int64 (position_bytes 4 or 8), batch rows of tokens
 *     contiguous values, position_stride apart (0: one row for all), negative
 *     ones allowed; NULL: start + token.
 *   1 ≤ dim ≤ 1024, rotated even, 2 ≤ rotated ≤ dim; batch · tokens ≤ 2^24. */
typedef struct muon_rotary {
  int64_t batch, tokens, dim, rotated;
  const double* freqs;
  const void* positions;
  int64_t position_stride, start;
  int32_t position_bytes;
  int32_t interleaved;
  float scale;
  int32_t dtype; /* muon_dtype_t */
} muon_rotary_t;

/* A tensor to turn: batch × tokens × heads × dim, strides {batch, token, head}.
 * out may be in itself (same address and strides). */
typedef struct muon_rotary_heads {
  const void* in;
  void* out;
  int64_t heads;
  int64_t in_strides[3], out_strides[3];
} muon_rotary_heads_t;

/* One or two tensors (queries and keys) in one launch. */
muon_status_t muon_rotary(const muon_rotary_t* rotary, const muon_rotary_heads_t* tensors, int32_t count,
                          void* stream);
/* Its gradient: the same with −θ, `in` the outputs' gradients. */
muon_status_t muon_rotary_grad(const muon_rotary_t* rotary, const muon_rotary_heads_t* tensors,
                               int32_t count, void* stream);

/* ----- dropout ------------------------------------------------------------ */

/* y = residual + x/(1 − p) where an element is kept, residual elsewhere.
 * Element i (row-major, i = row · cols + column) is kept where its random word
 * is at least p·2^32 rounded to a whole number: word i mod 4 of Philox4x32-10
 * with counter (i / 4, offset), 64 bits each, and key `seed`.  With
 * offset_device (one uint64 on the device, NULL: none) its value is added to
 * offset when the kernel runs, so that replays of a graph can differ.
 *   x, residual (NULL: none), y: rows × cols; 0 ≤ p ≤ 1 (1 keeps nothing).
 *   0 ≤ rows ≤ 2^24, 1 ≤ cols ≤ 2^20.
 * A dropped infinity or NaN leaves nothing.  y may be x or residual itself
 * (same address and stride). */
muon_status_t muon_dropout(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual,
                           double p, uint64_t seed, uint64_t offset, const uint64_t* offset_device,
                           void* y, int64_t ld_y, int64_t rows, int64_t cols, muon_dtype_t dtype,
                           void* stream);
/* Gradient of x: dy/(1 − p) where an element was kept, 0 elsewhere (the
 * residual's gradient is dy).  dx may be dy itself. */
muon_status_t muon_dropout_grad(const void* dy, int64_t ld_dy, double p, uint64_t seed, uint64_t offset,
                                const uint64_t* offset_device, void* dx, int64_t ld_dx, int64_t rows,
                                int64_t cols, muon_dtype_t dtype, void* stream);

/* ----- differential attention --------------------------------------------- */

/* Head h of `heads` has two maps, over the query heads 2h and 2h + 1 and the
 * key heads 2·(h / group) and 2·(h / group) + 1, group = heads / kv_heads:
 *   P_m = softmax over keys j of scale · q_m · k_m[j],
 *   out = (P_1 − lambda[h] · P_2) · v,  v of twice the width.
 *   q: batch × queries × 2·heads × dim;  k: batch × keys × 2·kv_heads × dim;
 *   v: batch × keys × kv_heads × 2·dim;  out: batch × queries × heads × 2·dim;
 *   lambda: heads float32 values; strides {batch, token, head}.
 *   causal ≠ 0: query i sees the keys j ≤ i + keys − queries (the last query
 *     the last key).  A query that sees no key gives zeros, and gradients 0,
 *     whatever it and its dout hold.
 *   sequences > 0: a packed batch (batch = 1, queries = keys = tokens): sequence
 *     i holds the tokens offsets[i] … offsets[i + 1] − 1 (sequences + 1 int32 on
 *     the device) and sees itself alone.  Tokens before the first and from the
 *     last offset on give zeros.  Offsets outside [0, tokens] are cut to it, one
 *     below its predecessor is raised to it.
 *   1 ≤ dim ≤ 128; kv_heads divides heads; 2^-60 ≤ scale ≤ 2^60 (and
 *   |q·k| ≤ 1e30 for the gradients);
 *   batch · queries, batch · keys ≤ 2^24; queries · group < 2^30;
 *   batch · queries · heads ≤ 2^28; at most 2^23 workgroups (per batch entry and
 *   key/value head one for 32 to 128 rows of queries · group, or 128 keys, and two
 *   and one per sequence more of a packed batch).
 * Keys behind the end of a sequence are never read.  Infinities and NaN of keys
 * and values that the causal rule hides from a row reach neither its result nor its
 * gradient, and those of a row's q and dout not the gradients of keys that it does
 * not see.
 * Tensors whose heads are not whole 16-byte chunks at 16-byte aligned addresses
 * (or with tokens 2^24 or more elements apart) are copied to the workspace. */
typedef struct muon_diff_attention {
  int64_t batch, queries, keys, heads, kv_heads, dim;
  const void* q;
  const void* k;
  const void* v;
  const float* lambda;
  int64_t q_strides[3], k_strides[3], v_strides[3];
  const int32_t* offsets;
  int64_t sequences;
  float scale;
  int32_t causal;
  int32_t dtype; /* muon_dtype_t */
} muon_diff_attention_t;

/* saved: NULL, or muon_diff_attention_saved_size bytes (256-byte aligned) that
 * receive what muon_diff_attention_grad reads: the maps' log-sums (fp32) and,
 * for MUON_DTYPE_F32, P_2 · v (fp32), for MUON_DTYPE_BF16 P_1 · v and P_2 · v
 * (16 bits a value with a scale per row: 2^-15 of the row's largest value). */
muon_status_t muon_diff_attention(const muon_diff_attention_t* attention, void* out,
                                  const int64_t out_strides[3], void* saved, size_t saved_bytes,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* Gradients of muon_diff_attention from the gradient of out, out itself (read
 * for MUON_DTYPE_F32 only) and `saved`.  With dA = dout·vᵀ, δ_m = Σ_j P_m · dA:
 *   dS_1 = P_1·(dA − δ_1), dS_2 = −lambda·P_2·(dA − δ_2),
 *   dq_m = scale·dS_m·k_m, dk_m = scale·Σ dS_mᵀ·q_m over the group's heads,
 *   dv = Σ (P_1 − lambda·P_2)ᵀ·dout over them, dlambda[h] = −Σ P_2·dA.
 *   dq, dk, dv have the shapes of q, k, v; dq, dlambda (heads float32 values) and
 *   the pair dk, dv may each be NULL: not wanted.
 * For MUON_DTYPE_BF16 A, dS and the probabilities are rounded to bf16 as operands
 * of the next product; scores, statistics and sums are fp32, dlambda is summed
 * from unrounded terms. */
typedef struct muon_diff_attention_grads {
  void* dq;
  void* dk;
  void* dv;
  float* dlambda;
  int64_t dq_strides[3], dk_strides[3], dv_strides[3];
} muon_diff_attention_grads_t;

muon_status_t muon_diff_attention_grad(const muon_diff_attention_t* attention, const void* dout,
                                       const int64_t dout_strides[3], const void* out,
                                       const int64_t out_strides[3], const void* saved, size_t saved_bytes,
                                       const muon_diff_attention_grads_t* grads, void* workspace,
                                       size_t workspace_bytes, void* stream);

/* Bytes of `saved`, and of the workspaces of muon_diff_attention (dout = NULL)
 * and muon_diff_attention_grad.  The addresses and strides of q, k, v and dout
 * decide whether room for their copies is needed; addresses are not read. */
muon_status_t muon_diff_attention_saved_size(const muon_diff_attention_t* attention, size_t* bytes);
muon_status_t muon_diff_attention_workspace_size(const muon_diff_attention_t* attention, const void* dout,
                                                 const int64_t dout_strides[3], size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* MUON_ATTENTION_H */
