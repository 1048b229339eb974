/*
 * dyra_layers.h - exact layers beside the approximated one of dyra.h: a dense
 * linear layer with its epilogue and its gradients, and a mixture-of-experts
 * layer for a few tokens.
 *
 * A model keeps some of its linear layers exact: at a few tokens per call the
 * approximated layer moves more bytes than the dense one. These are the
 * products such layers run, with what surrounds them fused in:
 *   dense    Z = X W^T + b, Y = act(Z) + R           (W: d_out x d_in)
 *            dZ = dY * act'(Z), dX = dZ W, dW = dZ^T X, db = column sums of dZ
 *   experts  logits = X Wr^T, the top_k experts of every token with softmax
 *            weights w, y = sum_k w_k Wd_e (act(Wg_e x) * (Wu_e x)) + r
 *
 * The conventions of dyra.h hold: dense row-major device matrices in the
 * handle's type, 16-byte aligned, owned by the caller; fp32 accumulation; work
 * enqueued on `stream`; a handle is bound to the device that was current when
 * it was created and is not used from two host threads or two streams at once
 * (its workspace is allocated at creation and never moves, so a captured call
 * may be replayed as long as the handle lives, under the same rule). Weights
 * are arguments of each call, never copied: a training step may change them
 * between calls. An output that overlaps an input or another output is refused
 * (DYRA_ERR_INVALID_ARG) except where said so.
 * No call throws; each returns DYRA_OK or a negative DYRA_ERR_* code and
 * enqueues nothing when it refuses its arguments.
 */
#ifndef DYRA_LAYERS_H_
#define DYRA_LAYERS_H_

#include "dyra.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct dyra_dense *dyra_dense_t;
typedef struct dyra_moe *dyra_moe_t;

/* Activations, in fp32 on the accumulated value. */
enum {
  DYRA_ACT_NONE = 0,
  DYRA_ACT_RELU = 1,
  DYRA_ACT_GELU = 2,      /* z Phi(z), Phi the normal distribution function */
  DYRA_ACT_GELU_TANH = 3, /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2 */
  DYRA_ACT_SILU = 4       /* z / (1 + exp(-z)) */
};

/*
 * A dense layer of d_in inputs and d_out outputs (1 .. 2^31 - 512). DYRA_BF16 needs both
 * to be multiples of 8 (16-byte rows), else DYRA_ERR_ALIGNMENT. *out is left
 * unchanged on error. The handle owns a workspace of a fixed size (see
 * dyra_dense_device_bytes), whatever the row counts of its calls.
 */
int dyra_dense_create(dyra_dense_t *out, int d_in, int d_out, dyra_dtype_t dtype);

/*
 * Z = X W^T + bias, Y = act(Z) + residual.
 *   X        : N x d_in
 *   W        : d_out x d_in
 *   bias     : d_out values, or NULL
 *   residual : N x d_out, or NULL; may be Y itself
 *   act      : DYRA_ACT_*
 *   Y        : N x d_out
 *   Z        : N x d_out, receives the pre-activations rounded to the layer's
 *              type (the Z of dyra_dense_backward), or NULL
 * Z is kept in fp32 inside the call: act and residual are applied before the
 * one rounding of Y. N == 0 is a no-op.
 * Errors: DYRA_ERR_INVALID_ARG (NULL handle, X, W or Y; N < 0 or > 2^31 - 512;
 * unknown act), DYRA_ERR_ALIGNMENT, DYRA_ERR_CUDA.
 */
int dyra_dense_forward(dyra_dense_t p, const void *X, const void *W, const void *bias,
                       const void *residual, int act, void *Y, void *Z, int64_t N,
                       dyra_stream_t stream);

/*
 * Gradients of dyra_dense_forward from dY, the gradient of Y (the gradient of
 * residual is dY itself):
 *   dZ = dY * act'(Z), dX = dZ W, dW = dZ^T X, dbias = column sums of dZ.
 *   dY    : N x d_out
 *   X, W  : as in the forward; X is needed for dW, W for dX, else NULL is taken
 *   Z     : the forward's pre-activations; not read for DYRA_ACT_NONE
 *   dZ    : N x d_out, receives dZ; needed unless act is DYRA_ACT_NONE (then
 *           dZ is dY and nothing is written here); may be dY or Z itself
 *   dX, dW, dbias : N x d_in, d_out x d_in, d_out; any of them may be NULL
 * The products use dZ rounded to the layer's type; dbias sums it unrounded.
 * The gradients overwrite what was there. With N == 0, dW and dbias are zero.
 * Sums run in a fixed order: equal calls give equal bits.
 * Errors as in the forward.
 */
int dyra_dense_backward(dyra_dense_t p, const void *dY, const void *X, const void *W,
                        const void *Z, int act, void *dZ, void *dX, void *dW, void *dbias,
                        int64_t N, dyra_stream_t stream);

/* Synchronise the device, then return and clear the device status bits
 * (DYRA_STATUS_* of dyra.h), or a negative error code. After a wait that ran out
 * (DYRA_STATUS_WAIT_TIMEOUT) results mean nothing until this has been called: it
 * makes the handle ready again. The same holds for dyra_moe_status. */
int dyra_dense_status(dyra_dense_t p);
size_t dyra_dense_device_bytes(dyra_dense_t p);
/* Free the handle (synchronises the device). NULL is a no-op. */
int dyra_dense_destroy(dyra_dense_t p);

/*
 * A mixture-of-experts layer: `experts` gated MLPs of d_model -> d_ff ->
 * d_model, of which each token uses top_k.
 *   1 <= d_model, d_ff <= DYRA_MOE_MAX_WIDTH (multiples of 8 for DYRA_BF16, else
 *   DYRA_ERR_ALIGNMENT)
 *   1 <= top_k <= experts, top_k <= DYRA_MOE_MAX_TOP_K, experts <= DYRA_MOE_MAX_EXPERTS
 *   act    : DYRA_ACT_*, the activation of the gate
 *   renorm : 1: a token's weights are the softmax over its top_k logits (they
 *            sum to one), 0: over all logits
 * Made for a few tokens, where a call is bound by reading the weights of the
 * experts that its tokens reach, once for every 64 tokens; larger N runs in
 * groups of 64 tokens.
 */
#define DYRA_MOE_MAX_TOP_K 16
#define DYRA_MOE_MAX_EXPERTS 512
#define DYRA_MOE_MAX_WIDTH (1 << 20)
int dyra_moe_create(dyra_moe_t *out, int d_model, int d_ff, int experts, int top_k, int act,
                    int renorm, dyra_dtype_t dtype);

/*
 * The router: for each of N tokens the top_k experts by logit, largest first
 * (equal logits: the lower index first; a NaN counts as the lowest logit), and
 * their weights. A softmax that a NaN logit takes part in gives NaN weights.
 *   X       : N x d_model
 *   Wr      : experts x d_model
 *   ids     : N x top_k int32 (output)
 *   weights : N x top_k float (output)
 * Logits are summed in fp64, where the products of the inputs are exact: they are
 * off by at most d_model 2^-53 of the sum of their products' magnitudes, and
 * experts closer than that may come in either order.
 */
int dyra_moe_route(dyra_moe_t p, const void *X, const void *Wr, int32_t *ids, float *weights,
                   int64_t N, dyra_stream_t stream);

/*
 * The experts, with given routing:
 *   Y[n] = sum over k of weights[n][k] Wd_e (act(Wg_e x_n) * (Wu_e x_n)) + residual[n],
 *   e = ids[n][k].
 *   ids      : N x top_k int32; an id outside 0 .. experts - 1 (e.g. -1) names no
 *              expert and adds nothing; a token may name an expert twice
 *   weights  : N x top_k float
 *   Wgu      : experts x 2 d_ff x d_model: each expert's gate rows, then its up rows
 *   Wd       : experts x d_model x d_ff
 *   residual : N x d_model, or NULL; may be Y itself
 *   Y        : N x d_model; a token without experts gets its residual, or zero
 * The hidden values are rounded to the layer's type, unweighted; everything
 * else is fp32 until the one rounding of Y. An expert's weights have no effect
 * on tokens that do not name it, whatever their values. Sums run in a fixed
 * order. N == 0 is a no-op.
 */
int dyra_moe_experts(dyra_moe_t p, const void *X, const int32_t *ids, const float *weights,
                     const void *Wgu, const void *Wd, const void *residual, void *Y, int64_t N,
                     dyra_stream_t stream);

/* The whole layer: dyra_moe_route, then dyra_moe_experts with its result. */
int dyra_moe_forward(dyra_moe_t p, const void *X, const void *Wr, const void *Wgu, const void *Wd,
                     const void *residual, void *Y, int32_t *ids, float *weights, int64_t N,
                     dyra_stream_t stream);

int dyra_moe_status(dyra_moe_t p);
size_t dyra_moe_device_bytes(dyra_moe_t p);
int dyra_moe_destroy(dyra_moe_t p);

#ifdef __cplusplus
}
#endif

#endif /* DYRA_LAYERS_H_ */
