/*
 * optimizer_b200.h -- C ABI of the weight update: one AdamW step over many tensors.
 *
 * The gradients are those of conv2d_backward_weight, conv1d_causal_backward and the like (a
 * gradient has its weight's layout).  The conventions of conv2d_b200.h hold: device pointers,
 * 16-byte aligned (the scales of 8-bit states: 4-byte), a stream, a status.
 *
 *     g = grad * *grad_scale
 *     m = beta1 * m + (1 - beta1) * g,   v = beta2 * v + (1 - beta2) * g^2
 *     p = p * (1 - lr * weight_decay) - lr * (m / (1 - beta1^step)) / (sqrt(v / (1 - beta2^step)) + eps)
 */
#ifndef OPTIMIZER_B200_H
#define OPTIMIZER_B200_H

#include "conv2d_b200.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One weight tensor, contiguous, with its states.
 *   param          : param_dtype; updated in place
 *   master         : NULL, or (param_dtype CONV_BF16) the fp32 weights: they are read and
 *                    updated, and param receives them rounded
 *   exp_avg, exp_avg_sq : m and v: fp32 (state_bits 32), or 8-bit codes (state_bits 8): e4m3
 *                    and e5m2 values in units of a scale, a power of two, for each 256 elements
 *   exp_avg_scale, exp_avg_sq_scale : (ceil(numel / 256),) fp32 for 8 bits, else NULL.  Fresh
 *                    states are codes 0 with scales 1.
 * A tensor without elements is passed over, whatever its other members hold. */
typedef struct {
    void *param;
    float *master;
    const void *grad;
    void *exp_avg;
    void *exp_avg_sq;
    float *exp_avg_scale;
    float *exp_avg_sq_scale;
    long long numel;
} adamw_tensor_t;

/* One step.  `tensors` is a HOST array of `count` entries, read before the call returns; the
 * tensors must not overlap.  Either all or none have master weights.
 *   step        : the step's number, 1 for the first; ignored where step_device is given
 *   step_device : NULL, or a device integer with that number, read when the kernel runs (for
 *                 a captured step, whose graph counts it up before each replay).  Below 1 the step changes nothing
 *                 and conv2d_sync_status reports CONV_ERR_INVALID_ARG.
 *   grad_scale  : NULL (1), or a device float that multiplies the gradients (the reciprocal
 *                 of a loss scale, a clipping coefficient).  Where it is not finite or not
 *                 above zero the step changes nothing.
 *   seed        : with 8-bit states, m and v are rounded up or down by chance, in proportion to
 *                 the distance (v moves too little a step for rounding to nearest).  The chance is
 *                 a fixed function of (seed, step, place in `tensors`, element): with
 *                 mix(h) = h ^ h >> 16, times 0x85EBCA6B, ^ >> 13, times 0xC2B2AE35, ^ >> 16 and all in 32 bits,
 *                 mix(element * 0x9E3779B1 + mix(mix(seed + 0x9E3779B9 * step) + 0x85EBCA77 * (place + 1))),
 *                 its low half for m, its high half for v.  A v above zero stays above zero.
 * A gradient that is not finite makes its own element's state NaN, no other's.
 * CONV_ERR_INVALID_ARG: count < 0, a NULL pointer, numel < 0, lr, eps or weight_decay negative
 * or not finite, a beta outside [0, 1), step < 1, state_bits other than 8 and 32, weights that
 * overlap; CONV_ERR_UNSUPPORTED: a misaligned pointer, or more than (2^31 - 1) * 1024 elements. */
int adamw_step(const adamw_tensor_t *tensors, int count, conv_dtype_t param_dtype, conv_dtype_t grad_dtype,
               int state_bits, double lr, double beta1, double beta2, double eps, double weight_decay,
               long long step, const long long *step_device, const float *grad_scale, unsigned seed,
               conv_stream_t stream);

/* The launches of a step, written into buf (buflen bytes, owned by the caller) as one JSON object: "master" (1: the
 * kernel with master weights), "batches" (1024 elements each, of a block), "launches": a list of {"first", "count"
 * (places in `tensors`), "blocks"}.  As if the device had `sms` SMs.  The pointers are checked as in
 * adamw_step, not read; nothing runs on a GPU.  CONV_ERR_INVALID_ARG also for a NULL or too small buffer. */
int adamw_describe_plan(const adamw_tensor_t *tensors, int count, conv_dtype_t param_dtype, int state_bits, int sms,
                        char *buf, size_t buflen);

#ifdef __cplusplus
}
#endif

#endif /* OPTIMIZER_B200_H */
