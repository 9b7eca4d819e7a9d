/*
 * lora_norm.h -- C ABI of the root-mean-square norm with the residual's addition, for the
 * inputs of lora_layer.h's layers (conventions as there).
 */
#ifndef LORA_NORM_H
#define LORA_NORM_H

#include <stdint.h>

#include "lora_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * For every row of x [T, K], with r the residual's row (0 without one):
 *     h = x + r,   y = h rsqrt( mean(h^2) + eps ) w
 * in fp32; each output is rounded once from fp32.
 *   x_dev, residual_dev    rows ldx and ldr elements apart; residual_dev may be NULL.
 *   weight_dev             w [K].
 *   residual_out_dev       h, rows ldr_out elements apart, or NULL; may be residual_dev or
 *                          x_dev itself (with the same row distance).
 *   y_dev                  y, dense [T, K], or NULL.
 *   xq_dev, sx_dev         y in e4m3, dense [T, K] bytes, and its row scales [T] fp32, or both
 *                          NULL: sx = max|y| / 448 (1 for a zero row) and xq = e4m3(y / sx),
 *                          nearest even, saturating, from the fp32 y; the row format of an e4m3 layer
 *                          (lora_forward_e4m3).
 *   dtype                  LORA_BF16 or LORA_F32: of x, the residual, w, h and y.
 * Rows need no alignment but their elements' (2 or 4 bytes; LORA_EINVAL without it): 16-byte
 * vectors are used where every pointer and row distance allows them.
 * Limits: 0 <= T <= 1 << 20, 1 <= K <= 32768, row distances >= K, eps >= 0; at least one of
 * y, xq, residual_out.  y, xq and sx overlap no input.  Errors: LORA_EINVAL, LORA_ECUDA.
 */
int lora_rms_norm(const void* x_dev, int ldx, const void* residual_dev, int ldr,
                  const void* weight_dev, float eps, int T, int K, int dtype,
                  void* residual_out_dev, int ldr_out, void* y_dev, void* xq_dev, float* sx_dev,
                  void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_NORM_H */
