/*
 * tp3d_rope.h - C ABI of the norm of query and key heads with the rotation by
 * position, forward and backward.  tp3d_paged.h has its form for a server
 * (tp3d_paged_rope_store).
 *
 * Row x (head_dim columns) of one head of the token at position p becomes
 *   n = x / sqrt(mean_c x_c^2 + eps) * w      (norm = 1; else n = x)
 *   y = R(p) n
 * where R(p) turns the pairs of the first rotary_dim columns and leaves the
 * others: pair j, of columns (j, j + rotary_dim / 2) or, interleaved, of
 * (2 j, 2 j + 1), by the angle p f_j, and multiplies it by `magnitude`:
 *   y_a = magnitude (n_a cos(p f_j) - n_b sin(p f_j)),
 *   y_b = magnitude (n_a sin(p f_j) + n_b cos(p f_j)).
 * The frequencies are given as turns per position in 64-bit fractions, so
 * that an angle is an integer product modulo one turn: exact for every
 * position an int32 holds, negative ones too.  Its cosine and sine are off by
 * 5 2^-24 of their own values at most.
 *
 * Ownership, streams and errors are those of tp3d.h.  Arithmetic is fp32;
 * results are rounded once.
 */
#ifndef TP3D_ROPE_H
#define TP3D_ROPE_H

#include "tp3d.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Frequencies f_j, j < rotary_dim / 2, from a base (10000, say), for a model
 * whose positions went up to `context` and are to go `factor` times as far:
 *   PLAIN   base^(-2 j / rotary_dim)
 *   LINEAR  the same over `factor`: positions are interpolated
 *   BASE    with base * factor^(rotary_dim / (rotary_dim - 2)): the last pair
 *           is interpolated, the first kept
 *   PARTS   pairs that make less than one turn over the context are
 *           interpolated, those of more than 32 turns kept, the share of the
 *           kept frequency growing linearly between; magnitude
 *           0.1 ln(factor) + 1 (else 1)                                      */
typedef enum {
  TP3D_ROPE_PLAIN = 0,
  TP3D_ROPE_LINEAR = 1,
  TP3D_ROPE_BASE = 2,
  TP3D_ROPE_PARTS = 3
} tp3d_rope_kind;

/* Writes turns[j] = f_j / (2 pi) * 2^64, rounded, and the magnitude, on the
 * host; the caller copies them to the device once.  PLAIN ignores `factor`,
 * all but PARTS `context`.  TP3D_EINVAL for a null pointer, an unknown kind, a
 * base, factor or context that is not finite or below 1, or BASE with a
 * rotary_dim of 2; TP3D_ESHAPE for a rotary_dim that is not even and
 * positive.                                                                  */
tp3d_status tp3d_rope_turns(int rotary_dim, double base, int kind, double factor, double context, uint64_t* turns,
                            float* magnitude);

/* How heads are normed and turned.
 *   dtype       of every array and of the weights: TP3D_BF16 or TP3D_F32
 *   head_dim    a multiple of 8, up to 256 (else TP3D_EUNSUPPORTED)
 *   rotary_dim  0, or a multiple of 16 up to head_dim (else TP3D_EUNSUPPORTED;
 *               above head_dim TP3D_ESHAPE)
 *   norm        0 or 1; without it eps and the weights are ignored
 *   magnitude   finite; eps finite, not negative (else TP3D_EINVAL)
 *   turns       rotary_dim / 2 words in device memory, 8-byte aligned
 *   q_weight, k_weight  head_dim elements each, 16-byte aligned, or NULL for
 *               ones                                                         */
typedef struct {
  int32_t dtype, head_dim, rotary_dim, interleaved, norm;
  float eps, magnitude;
  const uint64_t* turns;
  const void *q_weight, *k_weight;
} tp3d_rope;

/* (token, head) rows of head_dim contiguous columns, strides in elements; that
 * the rows of an output do not overlap is the caller's to keep.              */
typedef struct {
  int64_t token_stride, head_stride;
} tp3d_row_strides;

/* Q (tokens x heads) and K (tokens x kv_heads) rows normed and turned into
 * Q_out and K_out; positions: int32 of each token, in device memory.  Q_out may
 * be Q with the same strides, and K_out K (in place); other overlap of an output
 * with an input or output is TP3D_EOVERLAP.  Slices of the rows of one packed
 * product do not overlap.  heads, kv_heads >= 1, strides positive (else
 * TP3D_EINVAL), rows 16-byte aligned (else TP3D_EALIGN).                     */
tp3d_status tp3d_qk_rope(tp3d_ctx* ctx, const tp3d_rope* rope, int64_t tokens, int heads, int kv_heads, const void* Q,
                         tp3d_row_strides q_strides, const void* K, tp3d_row_strides k_strides,
                         const int32_t* positions, void* Q_out, tp3d_row_strides qo_strides, void* K_out,
                         tp3d_row_strides ko_strides, void* stream);

/* Backward: from the forward's inputs Q and K (used with norm = 1 only; else
 * they may be NULL) and the gradients dQ_out, dK_out of its results,
 *   g = R(p)^T dy,  s = 1 / sqrt(mean x^2 + eps),
 *   dx = s (w g - x s^2 mean(w g x)),  dw = sum over tokens and heads of g x s
 * into dQ, dK and dq_weight, dk_weight (head_dim elements of `dtype` each,
 * 16-byte aligned; NULL where they are not wanted; NULL without norm, else
 * TP3D_EINVAL).  Sums over tokens are fp32 in a fixed order, rounded once.
 * dQ may be dQ_out with the same strides (and dK dK_out).  `workspace`:
 * tp3d_qk_rope_bwd_workspace_bytes bytes, 256-byte aligned, contents free; NULL
 * where no weight's gradient is asked for.  With 0 tokens the weights'
 * gradients are zero.                                                        */
tp3d_status tp3d_qk_rope_bwd(tp3d_ctx* ctx, const tp3d_rope* rope, int64_t tokens, int heads, int kv_heads,
                             const void* Q, tp3d_row_strides q_strides, const void* K, tp3d_row_strides k_strides,
                             const int32_t* positions, const void* dQ_out, tp3d_row_strides dqo_strides,
                             const void* dK_out, tp3d_row_strides dko_strides, void* dQ, tp3d_row_strides dq_strides,
                             void* dK, tp3d_row_strides dk_strides, void* dq_weight, void* dk_weight, void* workspace,
                             void* stream);

/* Bytes of tp3d_qk_rope_bwd's workspace on the context's device (it does not
 * depend on the tokens); 0 for an invalid argument.                          */
size_t tp3d_qk_rope_bwd_workspace_bytes(tp3d_ctx* ctx, const tp3d_rope* rope);

#ifdef __cplusplus
}
#endif

#endif /* TP3D_ROPE_H */
