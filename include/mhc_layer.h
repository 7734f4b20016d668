/*
 * mhc_layer.h -- C ABI of the layer operators that stand between the mHC
 * aggregate and the mHC post (mhc_h_aggregate.h) on GB300 (sm_103a): RMS norm
 * with the residual's addition and an 8-bit output, matrix product with bias,
 * activation and residual, the gated product of a feed-forward, and rotary
 * positions, and of the model's end: the cross entropy of a product over a
 * vocabulary; each with its gradient.  Library: libmhc_layer.so.
 *
 * Storage types are BF16 and IEEE binary16 (mhc_dtype_t) and, for the 8-bit
 * output and operands, E4M3 (4 exponent bits, 3 mantissa bits, largest value
 * 448, no infinities).  Weights of the norm, biases, scales, frequencies,
 * rstd and the gradients of the norm's weight and of the bias are FP32.
 *
 * Rules shared by every call, as in mhc_h_aggregate.h: every data pointer is
 * a DEVICE pointer owned by the caller, aligned to its element; the library
 * allocates nothing and never synchronises; a call enqueues its kernels on
 * `stream` and returns.  T == 0 returns MHC_OK without launching (gradients
 * that are sums over tokens are written as zeros).  A NULL pointer where one
 * is required, a negative size, a stride smaller than its row, a misaligned
 * pointer, a size whose byte count overflows int64, a workspace that is too
 * small or an output that overlaps an input or another output returns
 * MHC_ERR_INVALID_ARG without launching; a size outside an operator's range
 * returns MHC_ERR_UNSUPPORTED; a failed launch MHC_ERR_CUDA
 * (mhc_layer_last_cuda_error() then has the code).
 *
 * Strides are in elements, between consecutive rows (tokens); rows themselves
 * are contiguous.
 *
 * Determinism.  Results do not depend on timing: repeated calls give
 * identical bytes, no operator uses floating-point atomics, and every sum has
 * a fixed order.  The norm's and rotary's outputs and the product's y, z and
 * grad_x (the gated product's among them) and a cross entropy's loss and lse
 * of a token depend only on that token's inputs and on the row sizes, not on
 * T: any split of the batch along T gives the same bytes.  (A cross entropy's
 * gradients depend on T.)
 */
#ifndef MHC_LAYER_H
#define MHC_LAYER_H

#include "mhc_h_aggregate.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Version of this ABI; changes when a declaration here changes in a way that a
 * caller compiled against it would notice (not when one is added). */
MHC_API int32_t mhc_layer_abi_version(void);

/* ---- RMS norm -------------------------------------------------------------
 *
 *   s[t,h]    = x[t,h] + residual[t,h]         (FP32; s = x without residual)
 *   rstd[t]   = 1 / sqrt( (sum over h of s^2) / H + eps )
 *   v[t,h]    = (s[t,h] * rstd[t]) * weight[h]
 *   total     = cvt(s)                          y = cvt(v)
 *
 * The norm is of the FP32 sum, not of its rounding.  x and residual have the
 * same storage type and row strides x_stride and residual_stride; total and y
 * are dense [T,H].  residual and total are given together or are both NULL.
 * rstd FP32 [T].  1 <= H <= 32768.
 */
MHC_API mhc_status_t mhc_rms_norm_fwd(const void* x, const void* residual, const float* weight,
                                      void* y, void* total, float* rstd, int64_t T, int64_t H,
                                      int64_t x_stride, int64_t residual_stride, float eps,
                                      mhc_dtype_t dtype, mhc_stream_t stream);

/* The same with an E4M3 output and FP32 scales, one per row (group == 0) or
 * per 128 channels (group == 128, the last group of a row may be shorter):
 *
 *   amax  = max over the group of |v|, at least 2^-60
 *   scale = amax / 448                y8 = e4m3( v * (448 / amax) )
 *
 * y8 E4M3 [T,H]; scale FP32 [T,G], G = 1 or ceil(H / 128); y8 * scale
 * approximates v.  A NaN in a group gives a NaN scale.
 */
MHC_API mhc_status_t mhc_rms_norm_fp8_fwd(const void* x, const void* residual, const float* weight,
                                          void* y8, float* scale, void* total, float* rstd,
                                          int64_t T, int64_t H, int64_t x_stride,
                                          int64_t residual_stride, float eps, int32_t group,
                                          mhc_dtype_t dtype, mhc_stream_t stream);

/* Gradients, from g (the gradient of y, row stride g_stride), s as the
 * forward stored it in total (or x, without residual; row stride s_stride),
 * its rstd and, optionally, the gradient that reaches total past the norm:
 *
 *   n[t,h]       = s[t,h] * rstd[t]           u[t,h] = g[t,h] * weight[h]
 *   m[t]         = (sum over h of u * n) / H
 *   grad_x[t,h]  = cvt( rstd[t] * (u[t,h] - n[t,h] * m[t]) + grad_total[t,h] )
 *   grad_weight[h] = sum over t of g[t,h] * n[t,h]
 *
 * grad_x [T,H] (of x and of the residual alike), grad_total dense [T,H] or
 * NULL, grad_weight FP32 [H].  workspace: mhc_rms_norm_bwd_workspace(T, H)
 * bytes, 16-byte aligned.
 */
MHC_API mhc_status_t mhc_rms_norm_bwd(const void* g, const void* s, const float* weight,
                                      const float* rstd, const void* grad_total, void* grad_x,
                                      float* grad_weight, void* workspace, int64_t workspace_bytes,
                                      int64_t T, int64_t H, int64_t g_stride, int64_t s_stride,
                                      mhc_dtype_t dtype, mhc_stream_t stream);

MHC_API int64_t mhc_rms_norm_bwd_workspace(int64_t T, int64_t H);

/* ---- Matrix product ---------------------------------------------------------
 *
 *   z[t,o] = (sum over i of x[t,i] * w[o,i]) (* x_scale[t] * w_scale[o]) + bias[o]
 *   y[t,o] = cvt( act(z[t,o]) + residual[t,o] )
 *
 * x [T,I] and w [O,I] of one type (row strides x_stride, w_stride); FP32
 * x_scale [T] and w_scale [O] with E4M3 operands, NULL with the others; bias
 * FP32 [O] or NULL; residual [T,O] of the output type (row stride
 * residual_stride) or NULL; y [T,O] of the output type, which is the
 * operands' own type unless they are E4M3; preact [T,O] or NULL takes cvt(z).
 * act: see mhc_activation_t; GELU is z * Phi(z), Phi the normal distribution.
 * Sums are FP32.  workspace: mhc_linear_workspace(...) bytes, 16-byte aligned
 * (0 when no operand has to be laid out again; see there).
 */
typedef enum mhc_activation {
    MHC_ACT_NONE = 0,
    MHC_ACT_RELU = 1,
    MHC_ACT_SILU = 2,
    MHC_ACT_GELU = 3
} mhc_activation_t;

MHC_API mhc_status_t mhc_linear_fwd(const void* x, const void* w, const float* bias,
                                    const void* residual, void* y, void* preact, void* workspace,
                                    int64_t workspace_bytes, int64_t T, int64_t I, int64_t O,
                                    int64_t x_stride, int64_t w_stride, int64_t residual_stride,
                                    mhc_activation_t act, mhc_dtype_t dtype, mhc_stream_t stream);

/* E4M3 operands; dtype is the type of residual, y and preact. */
MHC_API mhc_status_t mhc_linear_fp8_fwd(const void* x8, const float* x_scale, const void* w8,
                                        const float* w_scale, const float* bias,
                                        const void* residual, void* y, void* preact,
                                        void* workspace, int64_t workspace_bytes, int64_t T,
                                        int64_t I, int64_t O, int64_t x_stride, int64_t w_stride,
                                        int64_t residual_stride, mhc_activation_t act,
                                        mhc_dtype_t dtype, mhc_stream_t stream);

/* Gradients, from g (the gradient of y, dense [T,O]) and the forward's preact
 * (NULL when act is MHC_ACT_NONE):
 *
 *   u[t,o] = g[t,o] * act'(preact[t,o])
 *   grad_x[t,i] = cvt( sum over o of cvt(u[t,o]) * w[o,i] )     [T,I]
 *   grad_w[o,i] = cvt( sum over t of cvt(u[t,o]) * x[t,i] )     [O,I]
 *   grad_bias[o] = sum over t of u[t,o]                          FP32 [O]
 *
 * cvt(u) is what the products' 16-bit operands hold; grad_bias sums u itself.
 * Each of the three may be NULL and is then not computed.  (The residual's
 * gradient is g.)  x, w, g and preact are dense.  workspace:
 * mhc_linear_bwd_workspace(...) bytes, 16-byte aligned.
 */
MHC_API mhc_status_t mhc_linear_bwd(const void* g, const void* x, const void* w, const void* preact,
                                    void* grad_x, void* grad_w, float* grad_bias, void* workspace,
                                    int64_t workspace_bytes, int64_t T, int64_t I, int64_t O,
                                    mhc_activation_t act, mhc_dtype_t dtype, mhc_stream_t stream);

/* Workspace bytes of the product.  itemsize is 2 (BF16, binary16) or 1
 * (E4M3); strides and pointers' alignment decide whether an operand can be
 * read in place (rows that start on 16-byte boundaries), so the answer covers
 * the worst alignment of the pointers when aligned is 0, and 16-byte aligned
 * pointers when it is not 0. */
MHC_API int64_t mhc_linear_workspace(int64_t T, int64_t I, int64_t O, int64_t x_stride,
                                     int64_t w_stride, int32_t itemsize, int32_t aligned);
MHC_API int64_t mhc_linear_bwd_workspace(int64_t T, int64_t I, int64_t O, mhc_activation_t act,
                                         int32_t want_x, int32_t want_w, int32_t want_bias,
                                         int32_t aligned);

/* ---- Gated product -----------------------------------------------------------
 *
 * The first half of a gated feed-forward: both projections, the activation
 * and their product in one kernel.  w [2 F, I] holds the gate's rows 0 .. F-1
 * and the up projection's F .. 2 F-1:
 *
 *   z[t,j] = (sum over i of x[t,i] * w[j,i]) (* x_scale[t] * w_scale[j]) + bias[j]
 *   y[t,f] = cvt( act(z[t,f]) * z[t,F + f] )
 *
 * x [T,I] and w of one type (row strides x_stride, w_stride), scales FP32 [T]
 * and [2 F] with E4M3 operands; bias FP32 [2 F] or NULL; y [T,F]; preact
 * [T,2 F] or NULL takes cvt(z).  The types, the activations and the sums are
 * the product's; 2 F takes the place of O in its limits and in
 * mhc_linear_workspace(T, I, 2 F, ...), whose bytes workspace has.
 */
MHC_API mhc_status_t mhc_gated_linear_fwd(const void* x, const void* w, const float* bias, void* y,
                                          void* preact, void* workspace, int64_t workspace_bytes,
                                          int64_t T, int64_t I, int64_t F, int64_t x_stride,
                                          int64_t w_stride, mhc_activation_t act,
                                          mhc_dtype_t dtype, mhc_stream_t stream);

/* E4M3 operands; dtype is the type of y and preact. */
MHC_API mhc_status_t mhc_gated_linear_fp8_fwd(const void* x8, const float* x_scale, const void* w8,
                                              const float* w_scale, const float* bias, void* y,
                                              void* preact, void* workspace,
                                              int64_t workspace_bytes, int64_t T, int64_t I,
                                              int64_t F, int64_t x_stride, int64_t w_stride,
                                              mhc_activation_t act, mhc_dtype_t dtype,
                                              mhc_stream_t stream);

/* Gradients, from g (the gradient of y, dense [T,F]) and the forward's preact
 * (dense [T,2 F]; for every activation):
 *
 *   u[t,f]     = (g[t,f] * preact[t,F + f]) * act'(preact[t,f])
 *   u[t,F + f] = g[t,f] * act(preact[t,f])
 *   grad_x[t,i] = cvt( sum over j of cvt(u[t,j]) * w[j,i] )      [T,I]
 *   grad_w[j,i] = cvt( sum over t of cvt(u[t,j]) * x[t,i] )      [2 F,I]
 *   grad_bias[j] = sum over t of u[t,j]                           FP32 [2 F]
 *
 * cvt(u) is what the products' 16-bit operands hold; grad_bias sums u itself.
 * grad_w is summed in runs of at most 16384 tokens, which are added in FP32.
 * Each of the three may be NULL and is then not computed.  x and w have row
 * strides.  workspace: mhc_gated_linear_bwd_workspace(...) bytes, 16-byte
 * aligned; aligned as in mhc_linear_workspace.
 */
MHC_API mhc_status_t mhc_gated_linear_bwd(const void* g, const void* x, const void* w,
                                          const void* preact, void* grad_x, void* grad_w,
                                          float* grad_bias, void* workspace,
                                          int64_t workspace_bytes, int64_t T, int64_t I, int64_t F,
                                          int64_t x_stride, int64_t w_stride, mhc_activation_t act,
                                          mhc_dtype_t dtype, mhc_stream_t stream);

MHC_API int64_t mhc_gated_linear_bwd_workspace(int64_t T, int64_t I, int64_t F, int64_t x_stride,
                                               int64_t w_stride, int32_t want_x, int32_t want_w,
                                               int32_t want_bias, int32_t aligned);

/* ---- Cross entropy over a vocabulary -------------------------------------------
 *
 * The cross entropy of the logits z = x w^T with a target each, which are no
 * output and not kept for the gradients (those compute them again):
 *
 *   z[t,v]  = sum over i of x[t,i] * w[v,i]                       (FP32)
 *   lse[t]  = log( sum over v of exp(z[t,v]) )
 *   loss[t] = lse[t] - z[t,target[t]]
 *
 * x [T,I] and w [V,I] of one type (row strides x_stride, w_stride); target
 * int64 [T]; loss and lse FP32 [T].  A token whose target is outside 0 .. V-1
 * (negative, as -100, by custom) is ignored: its loss is 0; its lse is
 * computed all the same.  workspace:
 * mhc_linear_cross_entropy_workspace(...) bytes, 16-byte aligned: 8 bytes for
 * every 16 to 64 logits, or, with at most 8192 entries, 512 tokens and 2^19
 * logits of more than 1024 products each, their FP32 sums over runs of 1024
 * products (at most 1.4 of the operands' bytes).
 */
MHC_API mhc_status_t mhc_linear_cross_entropy_fwd(const void* x, const void* w,
                                                  const int64_t* target, float* loss, float* lse,
                                                  void* workspace, int64_t workspace_bytes,
                                                  int64_t T, int64_t I, int64_t V,
                                                  int64_t x_stride, int64_t w_stride,
                                                  mhc_dtype_t dtype, mhc_stream_t stream);

MHC_API int64_t mhc_linear_cross_entropy_workspace(int64_t T, int64_t I, int64_t V,
                                                   int64_t x_stride, int64_t w_stride,
                                                   int32_t aligned);

/* Gradients, from the gradients of loss and of lse (FP32 [T]; either may be
 * NULL, for zeros, not both) and the forward's lse.  With g[t] =
 * grad_loss[t], 0 for an ignored token:
 *
 *   d[t,v] = (g[t] + grad_lse[t]) * exp(z[t,v] - lse[t]) - (v == target[t] ? g[t] : 0)
 *   grad_x[t,i] = cvt( sum over v of cvt(d[t,v]) * w[v,i] )       [T,I]
 *   grad_w[v,i] = cvt( sum over t of cvt(d[t,v]) * x[t,i] )       [V,I]
 *
 * The logits are computed again and d is in the workspace by pieces of the
 * vocabulary (whole with at most 2^27 values, 256 MB); cvt(d) is d
 * rounded to the operands' type after a scaling (one for the whole call, a
 * power of two over the largest |g|, taken out again in FP32), so that
 * binary16 holds small probabilities and a g that all tokens share, as that of
 * a mean, is not rounded.  Sums over entries and over tokens are taken in runs
 * of at most 16384, which are added in FP32.  grad_x or grad_w may be NULL and
 * is then not computed.  A token without a gradient (g + grad_lse and g both
 * 0) has d = 0 whatever its logits; its x still enters grad_w as 0 * x, so
 * x must be finite there too.  workspace:
 * mhc_linear_cross_entropy_bwd_workspace(...) bytes, 16-byte aligned.
 */
MHC_API mhc_status_t mhc_linear_cross_entropy_bwd(const float* grad_loss, const float* grad_lse,
                                                  const void* x, const void* w,
                                                  const int64_t* target, const float* lse,
                                                  void* grad_x, void* grad_w, void* workspace,
                                                  int64_t workspace_bytes, int64_t T, int64_t I,
                                                  int64_t V, int64_t x_stride, int64_t w_stride,
                                                  mhc_dtype_t dtype, mhc_stream_t stream);

MHC_API int64_t mhc_linear_cross_entropy_bwd_workspace(int64_t T, int64_t I, int64_t V,
                                                       int64_t x_stride, int64_t w_stride,
                                                       int32_t want_x, int32_t want_w,
                                                       int32_t aligned);

/* ---- Rotary positions --------------------------------------------------------
 *
 * The first R values of each head are rotated in pairs by the angle
 * positions[t] * frequencies[j], j = 0 .. R/2 - 1; the rest are copied:
 *
 *   (a, b) -> cvt(a * c - b * s), cvt(b * c + a * s)
 *   c = magnitude * cos(angle)    s = magnitude * sin(angle)
 *
 * The pair j is (j, j + R/2) (half layout) or (2j, 2j + 1) (interleaved).
 * inverse != 0 rotates by -angle: the gradient, applied to the gradient of
 * out.  Frequencies scaled for long contexts are the caller's table; the
 * angle is reduced from the exact product, so positions of millions keep
 * their FP32 accuracy.
 *   x            in   dtype, T x heads x D with strides x_token, x_head: a
 *                     token's heads lie inside its stride (x_token at least
 *                     (heads - 1) x_head + D) or a head's tokens inside the
 *                     head's (x_head at least (T - 1) x_token + D)
 *   positions    in   int64 [T]
 *   frequencies  in   FP32 [R / 2]
 *   out          out  dtype, strides out_token, out_head, a token's heads
 *                     inside its stride; may be x itself (same pointer and
 *                     strides), and must otherwise not overlap it
 * 0 <= R <= D, R even, D <= 65536.
 */
MHC_API mhc_status_t mhc_rotary(const void* x, const int64_t* positions, const float* frequencies,
                                void* out, int64_t T, int64_t heads, int64_t D, int64_t R,
                                int64_t x_token, int64_t x_head, int64_t out_token,
                                int64_t out_head, float magnitude, int32_t interleaved,
                                int32_t inverse, mhc_dtype_t dtype, mhc_stream_t stream);

/* The cudaError_t value behind the last MHC_ERR_CUDA of this library on the
 * calling thread. */
MHC_API int32_t mhc_layer_last_cuda_error(void);

/* The kernels that wait for copies of their own (the products', the gated and
 * the cross entropy's among them, and the norm's for many rows of more than
 * 1024 values) bound every wait for a copy,
 * a free stage or a finished multiplication (1 s of the GPU's global timer), so no wait can hang
 * the GPU.  This returns 1 if a wait ran out on the current device since the
 * previous call, else 0, and clears the record; -1 if a CUDA call fails.  It
 * synchronizes the device.  A return of 1 means that the outputs of every
 * such call on the device since the previous call are invalid. */
MHC_API int64_t mhc_layer_wait_timeouts(void);

#ifdef __cplusplus
}
#endif

#endif /* MHC_LAYER_H */
