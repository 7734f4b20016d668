// What the layer library's translation units share: the calls from the entry
// points (mhc_layer.cu) to the launches of each operator.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mhc_launch.cuh"
#include "mhc_linear.cuh"
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
// kE4m3.  Every operand's rows start on 16-byte boundaries.
cudaError_t product(const linear::Product& p, int in, int out, cudaStream_t stream);
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
