/*
 * tcd_linear.h - C ABI of a layer's projections: what stands before and behind
 * the attention of tcd_cache.h in a model whose hidden states the constrained
 * decode step of tcd.h reads.
 *
 * A projection is a matrix product whose bias, activation, gate and residual
 * are applied where its sums are, so that each output is rounded and written
 * once:
 *
 *   z[i, o] = sum_k x[i, k] weight[o, k] + bias[o]
 *   y[i, o] = act(z[i, o]) + residual[i, o]                      without a gate
 *   g[i, o] = sum_k x[i, k] gate[o, k] + gate_bias[o]
 *   y[i, o] = act(g[i, o]) * z[i, o] + residual[i, o]            with a gate
 *
 * With a gate it is the first half of a gated feed-forward block; the second is
 * a projection back with the residual.
 *
 * Conventions are tcd.h's: the caller owns every buffer, calls are asynchronous
 * and capturable, argument errors are returned at once and launch nothing.
 * Calls are stateless and need no workspace: any number of them, captured or
 * not, may run at the same time as long as they write different memory.
 */
#ifndef TCD_LINEAR_H
#define TCD_LINEAR_H

#include "tcd_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations, of a value z in 32 bits. */
enum {
  TC_ACT_NONE = 0,
  TC_ACT_RELU = 1,      /* max(z, 0) */
  TC_ACT_SILU = 2,      /* z / (1 + exp(-z)) */
  TC_ACT_GELU = 3,      /* z / 2 (1 + erf(z / sqrt 2)) */
  TC_ACT_GELU_TANH = 4  /* z / 2 (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) */
};

#define TC_LINEAR_MAX_TOKENS (1 << 24)
#define TC_LINEAR_MAX_FEATURES (1 << 20)

/*
 * The weights of a projection.
 *
 *  device, dtype   the CUDA device and element type (TC_DT_BF16 or TC_DT_F16) of
 *                  everything in the call; calls run there.
 *  in_features, out_features   1 .. TC_LINEAR_MAX_FEATURES, odd ones among them.
 *  weight     (device) [out_features] rows of in_features elements,
 *             weight_stride elements apart (a multiple of 8, at least
 *             in_features), 16-byte aligned.
 *  gate       (device) the same for the gate, gate_stride apart; NULL: none.
 *  bias, gate_bias  (device) [out_features] or NULL (gate_bias: only with a gate).
 *  act        one of TC_ACT_*.
 */
typedef struct tc_linear_t {
  int32_t device;
  int32_t dtype;
  int32_t in_features;
  int32_t out_features;
  const void* weight;
  int64_t weight_stride;
  const void* gate;
  int64_t gate_stride;
  const void* bias;
  const void* gate_bias;
  int32_t act;
} tc_linear_t;

/*
 * tc_linear - a projection of n_tokens rows.
 *
 *  n_tokens  0 .. TC_LINEAR_MAX_TOKENS (0: nothing is launched).
 *  x         (device) rows of in_features elements, x_stride elements apart (a
 *            multiple of 8, at least in_features), 16-byte aligned.
 *  residual  (device) rows of out_features elements, residual_stride apart (any
 *            stride of at least out_features); NULL: none.  May be `out` itself
 *            (with the same stride), but must not overlap it in another way.
 *  out       (device) rows of out_features elements, out_stride apart (the same);
 *            must not overlap x, the weights or the biases (an overlap is
 *            refused; of rows with different strides, any that interleave).
 *  status    (device) one int32 that the caller has set to TC_OK: it becomes
 *            TC_ERR_DEVICE_TIMEOUT if a bounded wait of the kernel gave up (the
 *            outputs are then invalid), and is not written otherwise, so that
 *            one word may gather the errors of many calls.
 *
 * Sums, activation, product and residual are held in 32 bits and rounded once.
 * The order of a sum depends on the sizes and the GPU's number of SMs only: a call
 * gives the same bits each time, wherever its output and residual lie.
 */
typedef struct tc_linear_call_t {
  int32_t n_tokens;
  const void* x;
  int64_t x_stride;
  const void* residual;
  int64_t residual_stride;
  void* out;
  int64_t out_stride;
  int64_t wait_polls;  /* polls of one wait inside the kernel before it gives up; 0: the default (seconds) */
  int32_t withhold;    /* 0; tests: the kernel leaves out its first load, so that its waits run out */
} tc_linear_call_t;

tc_status tc_linear(const tc_linear_t* layer, const tc_linear_call_t* call, int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TCD_LINEAR_H */
