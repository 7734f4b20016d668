// What the layer library's translation units share: the calls from the entry
// points (mhc_layer.cu) to the launches of each operator.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mhc_launch.cuh"
#include "mhc_linear.cuh"
#include "mhc_linear_plan.h"
#include "mhc_norm.cuh"

namespace mhc {
namespace layer {

// SM count of the current device, used only to size grids (never the arithmetic).
int num_sms();

// RMS norm (mhc_launch_norm.cu).  out: norm::Out.
cudaError_t norm_fwd(const norm::FwdArgs& a, int dtype, int out, cudaStream_t stream);
cudaError_t norm_bwd(norm::BwdArgs a, float* grad_weight, float* workspace, int dtype, cudaStream_t stream);
uint32_t norm_bwd_partials(int64_t T, int64_t H);

// Rotary positions (mhc_launch_rotary.cu).
struct RotaryCall {
    const uint16_t* x;
    uint16_t* out;
    const int64_t* positions;
    const float* frequencies;
    int64_t T, heads, D, R;
    int64_t x_token, x_head, out_token, out_head;
    float magnitude;
    bool interleaved, inverse;
    int dtype;
    cudaStream_t stream;
};
cudaError_t rotary(const RotaryCall& c);

// Column sums of partial [P,H] (row pitch `pitch`) into out [H] (mhc_launch_norm.cu).
cudaError_t column_sum(const float* partial, float* out, uint32_t P, int64_t H, int64_t pitch, cudaStream_t stream);

// Matrix product (mhc_launch_linear.cu).  in, out: kBF16, kF16; in also
// kE4m3.  Every operand's rows start on 16-byte boundaries.  plan: plan_of's, or another.
cudaError_t product(const linear::Product& p, int in, int out, cudaStream_t stream);
cudaError_t product(const linear::Product& p, const linear::Plan& plan, int in, int out, cudaStream_t stream);
// An operand whose rows (`length` bytes, `stride` bytes apart) are copied to
// rows of `pitch` bytes (a multiple of 16).
struct RepackCall {
    const void* src;
    void* dst;
    int64_t rows, length, stride, pitch;
};
cudaError_t repack(const RepackCall* calls, int count, cudaStream_t stream);   // count 1 or 2
// u = g * act'(preact) (u, of row pitch `pitch`, null: not stored) and, with
// grad_bias, its column sums through `partial` (slope_partials(T) * O floats).
cudaError_t slope(const uint16_t* g, const uint16_t* preact, uint16_t* u, float* grad_bias, float* partial, int64_t T,
                  int64_t O, int64_t pitch, int act, int dtype, cudaStream_t stream);
int64_t slope_partials(int64_t T);
// p.e.y [M,N] = cvt(a^T b) (by *scale where scale is not null) with rows of both operands along m and n: a weight's
// gradient, stored a row a thread (mhc_launch_entropy.cu).
cudaError_t row_product(const linear::Product& p, const float* scale, int dtype, cudaStream_t stream);
// The same from sums [parts,M,N] over sum_plan's parts of K, tiles of their own.
cudaError_t apart_product(const linear::Product& p, float* sums, int dtype, cudaStream_t stream);

// The gated product (mhc_launch_gated.cu): p.b is w [2 F, I], p.N = 2 F.
cudaError_t gated_product(const linear::Product& p, int in, int out, cudaStream_t stream);
// u = [g up act'(gate) | g act(gate)] of preact [T, 2 F]; the rest as in slope, with 2 F columns.
cudaError_t gated_slope(const uint16_t* g, const uint16_t* preact, uint16_t* u, float* grad_bias, float* partial, int64_t T,
                        int64_t F, int64_t pitch, int act, int dtype, cudaStream_t stream);

// Cross entropy over a vocabulary (mhc_launch_entropy.cu).  The operands'
// rows start on 16-byte boundaries.
struct EntropyCall {
    const void* x;
    const void* w;
    const int64_t* target;
    int64_t T, I, V;
    int64_t x_stride, w_stride;
    int dtype;
    cudaStream_t stream;
};
// partial: entropy_pairs(T, V), at: T.
int64_t entropy_pairs(int64_t T, int64_t V);
cudaError_t entropy_fwd(const EntropyCall& c, float* loss, float* lse, float2* partial, float* at);
// The same through the logits' FP32 sums over the runs of K in memory (entropy_apart): sums [entropy_runs,T,V].
cudaError_t entropy_fwd_apart(const EntropyCall& c, float* loss, float* lse, float* sums);
// The gradients of loss and lse (either may be null), and where the logits' gradients leave what takes their scale out
// again: the factor `scale` of the products and sums below.
struct EntropyGrads {
    const float* loss;
    const float* lse;
    float* inverse;
};
// The gradient of `count` logits from `first` on, [T,count] at row pitch `pitch`.
cudaError_t entropy_logit_grad(const EntropyCall& c, const EntropyGrads& g, const float* lse, int64_t first, int64_t count,
                               uint16_t* d, int64_t pitch);
// That of all of them through such sums.
cudaError_t entropy_logit_grad_apart(const EntropyCall& c, const EntropyGrads& g, const float* lse, float* sums, uint16_t* d,
                                     int64_t pitch);
// grad_x += d w[first ..], in `parts` parts of the vocabulary (entropy_parts of a whole piece): onto sum_in [parts,T,I]
// (null: onto nothing), into sum_out or, where that is null (one part), scaled and rounded into grad_x.
uint32_t entropy_parts(int64_t T, int64_t I, int64_t count);
cudaError_t entropy_grad_x(const EntropyCall& c, const uint16_t* d, int64_t pitch, int64_t first, int64_t count, uint32_t parts,
                           const float* sum_in, float* sum_out, const float* scale, void* grad_x);
// grad_x from the parts' sums.
cudaError_t entropy_sum(const EntropyCall& c, const float* sums, uint32_t parts, const float* scale, void* grad_x);
cudaError_t entropy_grad_w(const EntropyCall& c, const uint16_t* d, int64_t pitch, int64_t first, int64_t count, const float* scale,
                           void* grad_w);

// The device address of the flag that these kernels set when a bounded wait
// runs out, for the current device.
cudaError_t timeouts_ptr(unsigned int** p);
// 1 if a bounded wait of these kernels ran out on the current device since the
// last call, else 0 (clears the record; synchronizes the device); -1 on a
// CUDA error.
int64_t take_wait_timeouts();

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace layer
}  // namespace mhc
