/*
 * hyena_nd_block.h -- the operators around the gated long convolution of a
 * block, on the same [B, C, n_1, ..., n_d] activations (part of
 * libhyena_nd.so; hyena_nd.h has the convolution and the status codes).
 *
 *   join     h = x + scale_c gate_bc m norm_post(y),  n = norm_pre(h): the
 *            residual join after a mixer, fused with the norms on both sides
 *            of it, the block's gate, the residual scale and dropout; and the
 *            norm alone, for the head of a stack.  Forward and backward.
 *   dropout  inverted dropout from a counter-based generator: the mask is a
 *            function of (seed, offset, element) and is never stored.
 *   ffn      the gated feed-forward block y = Wd (act(Wg x) * (Wu x)), taken
 *            over the channels at every position.  Forward and backward.
 *
 * Conventions, as in hyena_nd.h: device memory is the caller's; every call is
 * asynchronous on the given stream, allocates nothing and synchronises
 * nothing; argument errors are found on the host before anything is launched;
 * every device pointer is 16-byte aligned (the fp32 parameter vectors and the
 * generator state: 4 and 8 bytes); outputs may not overlap inputs or each
 * other.  Activations are contiguous, fp32 or bf16, arithmetic is fp32 and
 * each output is rounded once.  Results do not depend on the launch: sums
 * over positions run in a fixed order and no atomics are used.  Calls may be
 * captured into a graph.  A call whose `ws` is in use by another call on
 * another stream (or by another graph that may run at the same time) needs a
 * workspace of its own; workspaces need no initialisation.
 */
#ifndef HYENA_ND_BLOCK_H_
#define HYENA_ND_BLOCK_H_

#include "hyena_nd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations [B, C, L]: L is the product of the grid's extents, any length
 * from 1 (single tokens) on; B, C >= 1, B C L < 2^40, C <= 65536,
 * B L < 2^31, B C < 2^31.  With L = 1 a position's channels lie next to each other, so
 * token-major [T, C] activations are B = T, L = 1. */
typedef struct {
  int64_t B, C, L;
  hyena_nd_dtype io_dtype;
} hyena_nd_block_shape;

/* A norm over the channels of each position, with v the values there:
 *   RMS    vhat = v / sqrt(mean(v^2) + eps)
 *   LAYER  vhat = (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps)
 * and w_c vhat + b_c as its result.  w, b: device fp32 [C]; NULL stands for
 * ones and zeros.  NONE passes v on (w and b must then be NULL).
 * eps: finite and > 0 (not looked at with NONE). */
typedef enum { HYENA_ND_NORM_NONE = 0, HYENA_ND_NORM_RMS = 1, HYENA_ND_NORM_LAYER = 2 } hyena_nd_norm_kind;

typedef struct {
  hyena_nd_norm_kind kind;
  float eps;
  const float *w, *b;
} hyena_nd_norm;

/* The join of a block's output y to the residual stream x:
 *   h = x + scale_c gate_bc m norm_post(y)
 *   n = norm_pre(h)          (of the unrounded h; the next block's input)
 *   gate   device fp32 [B, C] or NULL (ones): the block's gate per sample
 *   scale  device fp32 [C] or NULL (ones): the residual scale
 *   p      dropout probability in [0, 1]; m is the factor of
 *          hyena_nd_dropout for the element's index in [B, C, L]
 *   rng    device int64 [2] (seed, offset), read when the kernels run; may be
 *          NULL where p rounds to no dropout. */
typedef struct {
  hyena_nd_norm post, pre;
  const float *gate, *scale;
  double p;
  const int64_t* rng;
} hyena_nd_join;

/* Gradients of the join's parameters, device fp32; NULL: not wanted. */
typedef struct {
  float *post_w, *post_b;   /* [C] */
  float *gate;              /* [B, C] */
  float *scale;             /* [C] */
  float *pre_w, *pre_b;     /* [C] */
} hyena_nd_join_grads;

/* n = norm(x).  kind NONE is HYENA_ND_ERR_INVALID_ARG. */
HYENA_ND_API hyena_nd_status hyena_nd_norm_forward(const hyena_nd_block_shape* s, const hyena_nd_norm* norm,
                                                   const void* x, void* n, void* cuda_stream);

/* dx (and dw, db, fp32 [C], each may be NULL) of n = norm(x) for dn = dL/dn.
 * The statistics are recomputed from x. */
HYENA_ND_API hyena_nd_status hyena_nd_norm_backward(const hyena_nd_block_shape* s, const hyena_nd_norm* norm,
                                                    const void* x, const void* dn, void* dx, float* dw, float* db,
                                                    void* ws, size_t ws_bytes, void* cuda_stream);

/* h and n of the join.  n must be NULL where pre.kind is NONE. */
HYENA_ND_API hyena_nd_status hyena_nd_join_forward(const hyena_nd_block_shape* s, const hyena_nd_join* j,
                                                   const void* x, const void* y, void* h, void* n,
                                                   void* cuda_stream);

/* Gradients of the join with respect to x, y and its parameters, given
 * dh = dL/dh (the part that reaches h past the norm; NULL: zero) and
 * dn = dL/dn (NULL exactly where pre.kind is NONE).  Everything else is
 * recomputed from x, y and the generator state, which must hold what it held
 * in the forward call.  With dht the whole gradient at h, per channel:
 *   dx = dht;  dy through the post norm of scale gate m dht;
 *   Q_bc = sum_l dht m yhat,  R_bc = sum_l dht m:
 *   dpost_w = sum_b scale gate Q,   dpost_b = sum_b scale gate R,
 *   dgate = scale (w Q + b R),      dscale = sum_b gate (w Q + b R). */
HYENA_ND_API hyena_nd_status hyena_nd_join_backward(const hyena_nd_block_shape* s, const hyena_nd_join* j,
                                                    const void* x, const void* y, const void* dh, const void* dn,
                                                    void* dx, void* dy, const hyena_nd_join_grads* grads, void* ws,
                                                    size_t ws_bytes, void* cuda_stream);

/* Workspace bytes of the two backward calls above; 0 if `s` is invalid. */
HYENA_ND_API size_t hyena_nd_join_workspace_bytes(const hyena_nd_block_shape* s);

/* Inverted dropout: y_i = x_i 65536 / (65536 - t) where lot_i >= t, else 0,
 * with t = floor(65536 p + 1/2) and 16-bit lots from Philox4x32-10 (Salmon et
 * al. 2011): element i of the flat tensor takes lot i % 8 of the counter
 * (i / 8, offset), key seed; lots 2w and 2w + 1 are the low and the high half
 * of word w.  A dropped element is 0 whatever its value (infinities and NaN
 * too).  t = 65536 drops everything.  The gradient of the call is the call
 * itself on dy with the same state.  rng: device int64 [2] (seed, offset),
 * read when the kernel runs, so that a captured call follows the state; NULL
 * is allowed where t = 0. */
HYENA_ND_API hyena_nd_status hyena_nd_dropout(const hyena_nd_block_shape* s, double p, const int64_t* rng,
                                              const void* x, void* y, void* cuda_stream);

/* The gated feed-forward block.  act: the gate's activation, SILU
 * g / (1 + exp(-g)) or GELU g Phi(g) (the normal distribution function).
 * Weights in the activations' dtype, row-major: Wg, Wu [F, C], Wd [C, F].
 * C and F: multiples of 8 up to 65536 (else HYENA_ND_ERR_UNSUPPORTED).
 * With bf16 the hidden values act(g) u, and in the gradients those of g and u
 * too, are rounded to bf16 once before the next product.  act and its slope
 * keep their relative accuracy where they are small, down to the smallest
 * normal number (the slope as a sum of its two terms).  With fp32 an infinity
 * in an operand or a hidden value gives NaN in what it reaches, and values
 * below 2^-110 are good to 2^-133. */
typedef enum { HYENA_ND_ACT_SILU = 0, HYENA_ND_ACT_GELU = 1 } hyena_nd_act;

typedef struct {
  hyena_nd_block_shape s;
  int64_t F;
  hyena_nd_act act;
} hyena_nd_ffn;

/* Workspace bytes of the forward (backward = 0) or backward (1) call; 0 if
 * the descriptor is invalid or unsupported. */
HYENA_ND_API size_t hyena_nd_ffn_workspace_bytes(const hyena_nd_ffn* f, int backward);

/* y = Wd (act(Wg x) * (Wu x)) at every position.  `control`: 256 bytes set up
 * by hyena_nd_workspace_init, whose status word takes device-side errors
 * (hyena_nd_device_status reads it); it may be shared by any calls. */
HYENA_ND_API hyena_nd_status hyena_nd_ffn_forward(const hyena_nd_ffn* f, const void* x, const void* wg,
                                                  const void* wu, const void* wd, void* y, void* control, void* ws,
                                                  size_t ws_bytes, void* cuda_stream);

/* Gradients for dy = dL/dy: dx as x, dwg, dwu, dwd as the weights (their
 * dtype too).  The hidden activations are recomputed, not stored. */
HYENA_ND_API hyena_nd_status hyena_nd_ffn_backward(const hyena_nd_ffn* f, const void* x, const void* wg,
                                                   const void* wu, const void* wd, const void* dy, void* dx,
                                                   void* dwg, void* dwu, void* dwd, void* control, void* ws,
                                                   size_t ws_bytes, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* HYENA_ND_BLOCK_H_ */
