/*
 * dan_train.h -- C ABI of the norms a model is trained through: what a forward
 * pass keeps for its gradient, and the gradients.
 *
 *   dan_ln_modulate_save       y = LayerNorm(x) * (1 + scale) + shift, the rows'
 *                              mean and 1/std, and x as an 8-bit checkpoint
 *   dan_ln_modulate_backward   dx, dscale and dshift, from x or its checkpoint
 *   dan_group_norm             group norm of channels-last images with an
 *                              activation, weight and bias, scale and shift per
 *                              image; the same two things kept on request
 *   dan_group_norm_backward    dx, dweight, dbias, dscale and dshift
 *
 * The conventions are those of dan.h (device pointers, 16-byte alignment unless
 * said otherwise, caller's stream, status codes, stream order, no allocation),
 * with these differences.
 *  - Results are not defined bit for bit.  Sums and statistics are held in fp32
 *    and each result is rounded once, to its own type.  A call's bits are the
 *    same every time (no atomics).  y, dx, the statistics, the checkpoints,
 *    and a group norm's dscale and dshift are batch invariant: a row's or
 *    image's bits do not depend on the others in the call (a group norm's
 *    follow from S, C, the groups, the type, and whether there is a checkpoint).
 *    dweight and dbias, and a LayerNorm's dscale and dshift, are sums over rows
 *    in an order that follows from the sizes and the GPU's SM count.
 *  - A call is one to four launches (gradients of parameters over more than 256
 *    images one more for each further factor of 256); one that cannot run whole
 *    launches none.
 *  - Not a number and infinities pass as the formulas have them: a row or group
 *    that holds one gives NaN, others are not touched.  Squares of differences
 *    are summed in fp32: a row or group whose sum leaves its range (differences
 *    of some 1e18 and more) is not normalised.
 *
 * Checkpoint of values v [rows, C] (C a multiple of 8): blocks of 32
 * neighbouring channels (the last one of a row may be shorter) share a power of
 * two 2^k, the least with k >= -126 at which no finite |v| of the block exceeds
 * 448 * 2^k; the code of a value is e4m3(v * 2^-k), nearest even (a NaN has a
 * NaN code; an infinity makes k = 120 and has the code of 448).  codes is
 * [rows, C] bytes, scales [rows, ceil(C / 32)] bytes that hold k + 127 (E8M0).
 * v * 2^-k is exact, so the checkpoint is defined bit for bit.  Both pointers
 * are needed or both NULL; codes must be 8-byte aligned, scales may lie
 * anywhere.
 */
#ifndef DAN_TRAIN_H
#define DAN_TRAIN_H

#include "dan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------- LayerNorm, kept for training
 * y[b,t,:] = bf16(n * (1 + scale) + shift), n = (x - mean) * rstd in fp32: the
 * formula whose gradient dan_ln_modulate_backward returns, rounded once (the
 * roundings that dan_ln_modulate puts between its steps are left out).  mean and
 * rstd = 1/sqrt(var + eps) are those of dan_ln_modulate, bit for bit, and stored
 * as stats [B*T, 2] fp32 (8-byte aligned).  codes, scales: the checkpoint of x,
 * or NULL.  Supported D, vec_bstride and y == x as for dan_ln_modulate. */
int dan_ln_modulate_save(const dan_bf16 *x, const dan_bf16 *scale, const dan_bf16 *shift,
                         int64_t vec_bstride, dan_bf16 *y, float *stats, uint8_t *codes,
                         uint8_t *scales, int64_t B, int64_t T, int64_t D, float eps, void *stream);
int dan_can_use_ln_modulate_save(const dan_bf16 *x, const dan_bf16 *scale, const dan_bf16 *shift,
                                 int64_t vec_bstride, const dan_bf16 *y, const float *stats,
                                 const uint8_t *codes, const uint8_t *scales, int64_t B, int64_t T,
                                 int64_t D, float eps);

/* The gradients.  With n = (x - mean) * rstd, g = dy * (1 + scale) and means
 * over a row's D columns:
 *   dx     = bf16(rstd * (g - mean(g) - n * mean(g * n)) [+ dres])
 *   dscale = bf16(sum over t of dy * n),  dshift = bf16(sum over t of dy)
 * x is [B, T, D] bf16, or NULL to take the values of the checkpoint codes and
 * scales (which are not looked at otherwise).  stats as dan_ln_modulate_save
 * stored them.  scale [B, D] with batch stride vec_bstride; dscale and dshift
 * [B, D] with batch stride grad_bstride (>= D, a multiple of 8), e.g. their
 * slices of the embedding's gradient.  dres [B, T, D] (or NULL): a gradient
 * that reaches x by another way, added before the rounding.  In place: dx == dy
 * or dx == dres.  T == 0 writes zeros to dscale and dshift.  B * D <= 2^30.
 * workspace: dan_ln_modulate_backward_workspace(B, T, D) bytes (0 for many short
 * batches), of the current device, 16-byte aligned, this call's alone until it has completed: two calls
 * that may run at the same time, or two captured graphs that may, need one
 * each. */
int64_t dan_ln_modulate_backward_workspace(int64_t B, int64_t T, int64_t D);
int dan_ln_modulate_backward(const dan_bf16 *dy, const dan_bf16 *x, const uint8_t *codes,
                             const uint8_t *scales, const float *stats, const dan_bf16 *scale,
                             int64_t vec_bstride, const dan_bf16 *dres, dan_bf16 *dx,
                             dan_bf16 *dscale, dan_bf16 *dshift, int64_t grad_bstride, int64_t B,
                             int64_t T, int64_t D, void *workspace, int64_t workspace_bytes,
                             void *stream);
int dan_can_use_ln_modulate_backward(const dan_bf16 *dy, const dan_bf16 *x, const uint8_t *codes,
                                     const uint8_t *scales, const float *stats,
                                     const dan_bf16 *scale, int64_t vec_bstride,
                                     const dan_bf16 *dres, const dan_bf16 *dx,
                                     const dan_bf16 *dscale, const dan_bf16 *dshift,
                                     int64_t grad_bstride, int64_t B, int64_t T, int64_t D,
                                     const void *workspace, int64_t workspace_bytes);

/* ------------------------------------------------------------------ group norm
 * x [N, S, C]: N images of S positions, channels last (a torch channels_last
 * [N, C, H, W] with S = H*W), of `type`.  A group is C / groups neighbouring
 * channels of one image at all its positions:
 *   n = (x - mean) * rstd,  rstd = 1/sqrt(var + eps)   (population variance)
 *   z = (n * weight + bias) * (1 + scale) + shift
 *   y = z, or z / (1 + exp(-z)) with act == DAN_SILU
 * weight and bias [C] of param_type (the type of x, or fp32; both or neither may
 * be NULL: 1 and 0); scale and shift [N, C] of `type` with image stride
 * vec_bstride (both or neither; a stride of whole 16 bytes).
 * stats: NULL, or [N, groups, 2] fp32 (mean, rstd).  codes, scales: NULL, or the
 * checkpoint of x, for C % 32 == 0 (with stats).  In place: y == x.
 * Supported: C % 8 == 0, C <= 2^20, groups a divisor of C,
 * lcm(C / groups, 8) <= 4096 (with a checkpoint lcm(C / groups, 32)),
 * S < 2^31, N < 2^28, N * groups < 2^31.  N == 0 or S == 0 launches nothing.
 * An image is one CTA's work at least (2 to 3 ns each on a GB300): hundreds of
 * thousands of images of some ten values each are better left to elementary
 * operations (882723 of 24 bf16 values take 2.2 ms, 0.6 so).
 * workspace: dan_group_norm_workspace(...) bytes, on the terms of
 * dan_ln_modulate_backward's; 0 bytes where a call needs none. */
typedef enum { DAN_BF16 = 0, DAN_FP16 = 1, DAN_FP32 = 2 } dan_type;
typedef enum { DAN_NO_ACT = 0, DAN_SILU = 1 } dan_act;

int64_t dan_group_norm_workspace(int64_t N, int64_t S, int64_t C, int64_t groups, int type,
                                 int checkpoint);
int dan_group_norm(const void *x, int type, const void *weight, const void *bias, int param_type,
                   const void *scale, const void *shift, int64_t vec_bstride, int act, void *y,
                   float *stats, uint8_t *codes, uint8_t *scales, int64_t N, int64_t S, int64_t C,
                   int64_t groups, float eps, void *workspace, int64_t workspace_bytes,
                   void *stream);
int dan_can_use_group_norm(const void *x, int type, const void *weight, const void *bias,
                           int param_type, const void *scale, const void *shift,
                           int64_t vec_bstride, int act, const void *y, const float *stats,
                           const uint8_t *codes, const uint8_t *scales, int64_t N, int64_t S,
                           int64_t C, int64_t groups, float eps, const void *workspace,
                           int64_t workspace_bytes);

/* The gradients.  With dz = dy (times the derivative of SiLU at z),
 * a = weight * (1 + scale), sums over an image's positions
 *   s0 = sum dz,  s1 = sum dz * n                      (per image and channel)
 * and means over a group's S * C / groups values:
 *   dx      = rstd * (a * dz - mean(a * dz) - n * mean(a * dz * n))
 *   dweight = sum over images of (1 + scale) * s1,  dbias = ... (1 + scale) * s0
 *   dscale  = weight * s1 + bias * s0,  dshift = s0
 * x is [N, S, C] of `type`, or NULL to take the values of the checkpoint codes
 * and scales (C % 32 == 0).  dx has `type`, dweight and dbias [C] param_type,
 * dscale and dshift [N, C] `type` with image stride grad_bstride; each pair is
 * there when its parameters are.  In place: dx == dy.  S == 0 writes zeros to
 * dscale and dshift, N * S == 0 to dweight and dbias, whatever the parameters are.
 * workspace: dan_group_norm_backward_workspace(...) bytes, on the same terms. */
int64_t dan_group_norm_backward_workspace(int64_t N, int64_t S, int64_t C, int64_t groups, int type,
                                          int checkpoint);
int dan_group_norm_backward(const void *dy, const void *x, int type, const uint8_t *codes,
                            const uint8_t *scales, const float *stats, const void *weight,
                            const void *bias, int param_type, const void *scale, const void *shift,
                            int64_t vec_bstride, int act, void *dx, void *dweight, void *dbias,
                            void *dscale, void *dshift, int64_t grad_bstride, int64_t N, int64_t S,
                            int64_t C, int64_t groups, void *workspace, int64_t workspace_bytes,
                            void *stream);
int dan_can_use_group_norm_backward(const void *dy, const void *x, int type, const uint8_t *codes,
                                    const uint8_t *scales, const float *stats, const void *weight,
                                    const void *bias, int param_type, const void *scale,
                                    const void *shift, int64_t vec_bstride, int act,
                                    const void *dx, const void *dweight, const void *dbias,
                                    const void *dscale, const void *dshift, int64_t grad_bstride,
                                    int64_t N, int64_t S, int64_t C, int64_t groups,
                                    const void *workspace, int64_t workspace_bytes);

#ifdef __cplusplus
}
#endif

#endif /* DAN_TRAIN_H */
