/*
 * muon_layers.h — the layers whose gradients the Muon step consumes, in the
 * same library as muon_ns.h (libmuon_ns.so), for MI355X (gfx950):
 *
 *   muon_embedding   lookup with scaling; its gradient by sorted tokens
 *   muon_rms_norm    root-mean-square norm with the residual's addition
 *   muon_gated_ffn   gated feed-forward block (two projections, activation
 *                    and product in one kernel, then the down projection)
 *
 * each with its backward pass.  Conventions are those of muon_ns.h: device
 * pointers owned by the caller, work enqueued asynchronously on `stream`
 * (kernel launches only, so a call can be captured into a graph), every
 * argument checked on the host before anything is enqueued, status codes
 * with muon_last_error(), MUON_DEBUG_SYNC=1, no C++ exception across the
 * boundary, 256-byte aligned caller-allocated workspaces that overlap no
 * tensor of the call.  These calls use `stream` alone and record nothing for
 * muon_profile_read.  They add entry points only: MUON_NS_ABI_VERSION is
 * unchanged.
 *
 * Shared by every entry point:
 *   - matrices are row-major with rows of contiguous elements and a row
 *     stride `ld_*` ≥ the row length, in elements.  Any stride and any
 *     alignment of the element type is accepted.  Rows of whole aligned
 *     16-byte chunks are the fast case; others take unaligned accesses and
 *     single elements at a row's end (or, for the bf16 feed-forward products
 *     of more than a few tokens, one aligned copy in the workspace).
 *   - dtype is MUON_DTYPE_F32 or MUON_DTYPE_BF16.  Arithmetic, sums and
 *     statistics are fp32; an output is rounded once, when it is stored.
 *   - sums run in a fixed order that depends on the sizes alone: equal calls
 *     give equal bits.
 *   - an output may not overlap an input or another output unless the entry
 *     point says so (MUON_ERR_ALIAS); overlap is judged by the address ranges
 *     from a tensor's first to its last element.
 *   - 0 ≤ tokens ≤ 2^24; 1 ≤ vocab ≤ 2^24; dim, model and hidden are
 *     1 … 2^20; strides are at most 2^32 elements.  With zero tokens nothing is read; gradients of weights are still written.
 */
#ifndef MUON_LAYERS_H
#define MUON_LAYERS_H

#include "muon_ns.h"

#ifdef __cplusplus
extern "C" {
#endif

/* out[t] = scale · weight[ids[t]] for t < tokens; a row of zeros where
 * ids[t] is outside [0, vocab) (padding).
 *   ids: int32 (id_bytes = 4) or int64 (id_bytes = 8), contiguous;
 *   weight: vocab × dim, out: tokens × dim, both `dtype`; scale finite. */
muon_status_t muon_embedding(const void* ids, int32_t id_bytes, int64_t tokens, const void* weight,
                             int64_t ld_weight, int64_t vocab, int64_t dim, float scale, void* out,
                             int64_t ld_out, muon_dtype_t dtype, void* stream);

/* dweight[v] = scale · Σ_{t: ids[t] = v} dy[t], zero rows for ids that do
 * not occur; with accumulate ≠ 0 the sum is added to dweight instead and the
 * other rows are neither read nor written.  Token ids outside [0, vocab)
 * contribute nothing.
 *   dy: tokens × dim of `dtype`; dweight: vocab × dim of `dweight_dtype`.
 * The tokens are sorted by id (stable), each run of equal ids is summed in
 * token order (long runs in pieces of 16 sorted positions). */
muon_status_t muon_embedding_grad(const void* dy, int64_t ld_dy, const void* ids, int32_t id_bytes,
                                  int64_t tokens, int64_t vocab, int64_t dim, float scale,
                                  void* dweight, int64_t ld_dweight, muon_dtype_t dtype,
                                  muon_dtype_t dweight_dtype, int32_t accumulate, void* workspace,
                                  size_t workspace_bytes, void* stream);
muon_status_t muon_embedding_grad_workspace_size(int64_t tokens, int64_t vocab, int64_t dim,
                                                 size_t* bytes);

/* s = x + residual (fp32; s = x without residual)
 * rstd[t] = 1 / √(mean_j s[t][j]² + eps),  y = s · rstd · weight.
 *   x, residual (NULL: none), y, sum: tokens × dim of `dtype`; weight: dim
 *   values of `weight_dtype`; rstd: tokens float32 (NULL: not wanted).
 *   sum receives s rounded to dtype (NULL: not wanted; only with residual).
 *   y uses s before that rounding.  eps ≥ 0 finite (with eps = 0 a row of
 *   zeros gives NaN, as the formula does).
 * y or sum may be x or residual itself (same address and stride). */
muon_status_t muon_rms_norm(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual,
                            const void* weight, muon_dtype_t weight_dtype, float eps, void* y,
                            int64_t ld_y, void* sum, int64_t ld_sum, float* rstd, int64_t tokens,
                            int64_t dim, muon_dtype_t dtype, void* stream);

/* Backward of muon_rms_norm.  With n = s·rstd and c = mean_j(weight·dy·n):
 *   dx = rstd·(weight·dy − n·c) + dsum   (the gradient of x and of residual)
 *   dweight = Σ_t dy[t]·n[t]             (added to dweight if accumulate ≠ 0)
 *   s: the sum muon_rms_norm wrote (x without residual); rstd as it wrote it;
 *   dsum: gradient reaching the sum by other ways (NULL: none).
 *   dweight (NULL: not wanted): dim values of weight_dtype.
 * dx may be dy or dsum itself (same address and stride). */
muon_status_t muon_rms_norm_grad(const void* dy, int64_t ld_dy, const void* s, int64_t ld_s,
                                 const void* weight, muon_dtype_t weight_dtype, const float* rstd,
                                 const void* dsum, int64_t ld_dsum, void* dx, int64_t ld_dx,
                                 void* dweight, int32_t accumulate, int64_t tokens, int64_t dim,
                                 muon_dtype_t dtype, void* workspace, size_t workspace_bytes,
                                 void* stream);
muon_status_t muon_rms_norm_grad_workspace_size(int64_t tokens, int64_t dim, size_t* bytes);

typedef enum muon_activation {
  MUON_ACT_SILU = 0,     /* v / (1 + e^-v)                                   */
  MUON_ACT_GELU = 1,     /* v · Φ(v), Φ the normal distribution function     */
  MUON_ACT_GELU_TANH = 2 /* its tanh form, coefficients √(2/π) and 0.044715  */
} muon_activation_t;

/* The block's sizes and weights.
 *   w_gate, w_up: hidden × model; w_down: model × hidden (torch Linear
 *   layout: out_features × in_features), all of `dtype`. */
typedef struct muon_ffn {
  int64_t tokens, model, hidden;
  const void* w_gate;
  const void* w_up;
  const void* w_down;
  int64_t ld_gate, ld_up, ld_down;
  int32_t dtype;      /* muon_dtype_t */
  int32_t activation; /* muon_activation_t */
} muon_ffn_t;

/* g = x·w_gateᵀ, u = x·w_upᵀ, h = act(g)·u, y = h·w_downᵀ.
 *   x, y: tokens × model of dtype.
 *   saved: NULL, or muon_gated_ffn_saved_size bytes (256-byte aligned) that
 *   receive what muon_gated_ffn_grad reads: h in dtype, and the factors
 *   a = u·act'(g) and b = act(g) — float32 for MUON_DTYPE_F32; for
 *   MUON_DTYPE_BF16 the upper 24 bits of the float32 values (its whole range,
 *   errors below 2^-15 relative), since their products are rounded again.
 * g and u are never rounded before h; h, an operand of the next product, is
 * rounded to dtype. */
muon_status_t muon_gated_ffn(const muon_ffn_t* ffn, const void* x, int64_t ld_x, void* y,
                             int64_t ld_y, void* saved, size_t saved_bytes, void* workspace,
                             size_t workspace_bytes, void* stream);

/* Gradients of muon_gated_ffn from dy (tokens × model) and `saved`:
 *   dh = dy·w_down, dg = dh·a, du = dh·b (rounded to dtype),
 *   dx = dg·w_gate + du·w_up,
 *   dw_gate = dgᵀ·x, dw_up = duᵀ·x, dw_down = dyᵀ·h.
 *   dx (NULL: not wanted): tokens × model of dtype; the weight gradients (all
 *   three, or all NULL: not wanted) have the weights' shapes and are
 *   grad_dtype; with accumulate ≠ 0 they are added to what is there.
 * ffn->activation is not read (its derivative is in `saved`). */
typedef struct muon_ffn_grads {
  void* dx;
  void* dw_gate;
  void* dw_up;
  void* dw_down;
  int64_t ld_dx, ld_gate, ld_up, ld_down;
  int32_t grad_dtype; /* muon_dtype_t of the three weight gradients */
  int32_t accumulate;
} muon_ffn_grads_t;

muon_status_t muon_gated_ffn_grad(const muon_ffn_t* ffn, const void* x, int64_t ld_x,
                                  const void* dy, int64_t ld_dy, const void* saved,
                                  size_t saved_bytes, const muon_ffn_grads_t* grads,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of `saved`, and of the workspaces of muon_gated_ffn (grad = 0) and
 * muon_gated_ffn_grad (grad = 1).  ffn->activation is not read.  For bf16 the
 * workspace has room for aligned copies of x and dy, and of each weight whose
 * address, stride and row length do not give 16-byte aligned rows of whole
 * 16-byte chunks; `saved` does not depend on that. */
muon_status_t muon_gated_ffn_saved_size(const muon_ffn_t* ffn, size_t* bytes);
muon_status_t muon_gated_ffn_workspace_size(const muon_ffn_t* ffn, int32_t grad, size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* MUON_LAYERS_H */
