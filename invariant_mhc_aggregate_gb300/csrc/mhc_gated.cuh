// The first pass of the gated product's gradients (definitions in
// mhc_layer.h).
#pragma once

#include "mhc_linear.cuh"

namespace mhc {
namespace gated {

// u = [g up act'(gate) | g act(gate)] over [T, 2 F], rounded to u (row pitch
// `pitch`; null: not stored), and the column sums of the unrounded u over each
// of gridDim.y runs of `rows` rows in partial [gridDim.y, 2 F] (null: not
// wanted).  Block (32, 8): 32 W columns of each half, 8 rows at a time.
// HBM-bound: 10 bytes a value of g, T = 4096, F = 7168 44 us (6.7 TB/s; 48 with the
// column sums).
template <int DT, int W, int ACT>
__global__ void __launch_bounds__(32 * linear::kSlopeRows, 3)
slope_kernel(const uint16_t* __restrict__ g, const uint16_t* __restrict__ preact, uint16_t* __restrict__ u,
             float* __restrict__ partial, int64_t T, int64_t F, int64_t pitch, int64_t rows) {
    using namespace linear;
    pdl_enter();
    __shared__ float part[kSlopeRows][32 * W];
    const int64_t c = (int64_t(blockIdx.x) * 32 + threadIdx.x) * W;
    const int64_t t0 = int64_t(blockIdx.y) * rows, t1 = min(t0 + rows, T);
    float sum_gate[W], sum_up[W];
#pragma unroll
    for (int i = 0; i < W; ++i) sum_gate[i] = sum_up[i] = 0.0f;
    for (int64_t t = t0 + threadIdx.y; t < t1 && c < F; t += kSlopeRows) {
        Row<W> gr, gate, up;
        gr.load(g + t * F + c);
        gate.load(preact + t * 2 * F + c);
        up.load(preact + t * 2 * F + F + c);
        float a[W], b[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float gv = gr.template value<DT>(i), z = gate.template value<DT>(i);
            a[i] = __fmul_rn(__fmul_rn(gv, up.template value<DT>(i)), slope<ACT>(z));
            b[i] = __fmul_rn(gv, activation<ACT>(z));
            sum_gate[i] = __fadd_rn(sum_gate[i], a[i]);
            sum_up[i] = __fadd_rn(sum_up[i], b[i]);
        }
        if (u != nullptr) {
            store_row<DT>(u + t * pitch + c, a);
            store_row<DT>(u + t * pitch + F + c, b);
        }
    }
    if (partial == nullptr) return;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        if (half == 1) __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) part[threadIdx.y][threadIdx.x * W + i] = half == 0 ? sum_gate[i] : sum_up[i];
        __syncthreads();
        for (int i = threadIdx.y * 32 + threadIdx.x; i < 32 * W; i += 32 * kSlopeRows) {
            const int64_t f = int64_t(blockIdx.x) * 32 * W + i;
            if (f < F) {
                float s = part[0][i];
#pragma unroll
                for (int y = 1; y < kSlopeRows; ++y) s = __fadd_rn(s, part[y][i]);
                partial[int64_t(blockIdx.y) * 2 * F + half * F + f] = s;
            }
        }
    }
}

}  // namespace gated
}  // namespace mhc
