// Matrix product kernels (sm_103a): C[m,n] = sum over k of A[m,k] * B[n,k],
// with scales, bias, activation and residual applied to the FP32 sum before
// its one rounding.  Definitions in mhc_layer.h.  The forward is (m, n, k) =
// (t, o, i), grad_x (t, i, o) and grad_w (o, i, t).
#pragma once

#include <cuda_fp8.h>

#include "mhc_device.cuh"

namespace mhc {
namespace linear {

constexpr int kE4m3 = 2;   // operand type, beside kBF16 and kF16

enum Act { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3 };

__device__ __forceinline__ float activation(float z, int act) {
    switch (act) {
        case kActRelu: return z * (z > 0.0f ? 1.0f : 0.0f);
        case kActSilu: return __fdividef(z, 1.0f + __expf(-z));
        case kActGelu: return 0.5f * z * (1.0f + erff(z * 0.70710678f));
        default: return z;
    }
}

__device__ __forceinline__ float slope(float z, int act) {
    switch (act) {
        case kActRelu: return z > 0.0f ? 1.0f : 0.0f;
        case kActSilu: {
            const float p = 1.0f / (1.0f + expf(-z));
            return p * (1.0f + z * (1.0f - p));
        }
        case kActGelu: return 0.5f * (1.0f + erff(z * 0.70710678f)) + z * expf(-0.5f * z * z) * 0.39894228f;
        default: return 1.0f;
    }
}

struct Epilogue {
    const float* row_scale;      // [M] and col_scale [N]: E4M3 operands only, else null
    const float* col_scale;
    const float* bias;           // [N] or null
    const uint16_t* residual;    // [M,N], row stride residual_stride, or null
    uint16_t* y;                 // [M,N]
    uint16_t* preact;            // [M,N] or null
    int64_t residual_stride;
    int act;
};

struct Product {
    const void* a;
    const void* b;
    int64_t a_m, a_k, b_n, b_k;   // strides in elements; one of each pair is 1
    int64_t M, N, K;
    Epilogue e;
};

template <int IN>
__device__ __forceinline__ float operand(const void* p, int64_t i) {
    if constexpr (IN == kE4m3) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(p)[i], __NV_E4M3);
        return __half2float(__half(h));
    } else {
        return Elem<IN>::one(static_cast<const uint16_t*>(p)[i]);
    }
}

template <int OUT>
__device__ __forceinline__ void finish(const Epilogue& e, int64_t N, int64_t m, int64_t n, float sum) {
    float z = sum;
    if (e.row_scale != nullptr) z = z * e.row_scale[m] * e.col_scale[n];
    if (e.bias != nullptr) z += e.bias[n];
    if (e.preact != nullptr) e.preact[m * N + n] = Elem<OUT>::cvt(z);
    z = activation(z, e.act);
    if (e.residual != nullptr) z += Elem<OUT>::one(e.residual[m * e.residual_stride + n]);
    e.y[m * N + n] = Elem<OUT>::cvt(z);
}

// 64 x 64 tiles, 16 of k at a time through shared memory, 4 x 4 sums a thread.
template <int IN, int OUT>
__global__ void __launch_bounds__(256) simple_kernel(const Product p) {
    pdl_enter();
    __shared__ float sa[16][65], sb[16][65];
    const int64_t m0 = int64_t(blockIdx.y) * 64, n0 = int64_t(blockIdx.x) * 64;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < p.K; k0 += 16) {
        for (int i = threadIdx.x; i < 1024; i += 256) {
            const int ka = p.a_k == 1 ? i % 16 : i / 64, ma = p.a_k == 1 ? i / 16 : i % 64;
            sa[ka][ma] = k0 + ka < p.K && m0 + ma < p.M ? operand<IN>(p.a, (m0 + ma) * p.a_m + (k0 + ka) * p.a_k) : 0.0f;
            const int kb = p.b_k == 1 ? i % 16 : i / 64, nb = p.b_k == 1 ? i / 16 : i % 64;
            sb[kb][nb] = k0 + kb < p.K && n0 + nb < p.N ? operand<IN>(p.b, (n0 + nb) * p.b_n + (k0 + kb) * p.b_k) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += sa[k][ty + 16 * i] * sb[k][tx + 16 * j];
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m < p.M && n < p.N) finish<OUT>(p.e, p.N, m, n, acc[i][j]);
        }
}

// u = g * act'(preact) over [T,O], rounded to u (null: not stored), and the
// column sums of the unrounded u over each of gridDim.y runs of `rows` rows
// in partial [gridDim.y, O] (null: not wanted).  Block (32, 8): 32 W columns,
// 8 rows at a time.
constexpr int kSlopeRows = 8;

template <int DT, int W>
__global__ void __launch_bounds__(32 * kSlopeRows)
slope_kernel(const uint16_t* __restrict__ g, const uint16_t* __restrict__ preact, uint16_t* __restrict__ u,
             float* __restrict__ partial, int64_t T, int64_t O, int64_t rows, int act) {
    pdl_enter();
    __shared__ float part[kSlopeRows][32 * W];
    const int64_t c = (int64_t(blockIdx.x) * 32 + threadIdx.x) * W;
    const int64_t t0 = int64_t(blockIdx.y) * rows, t1 = min(t0 + rows, T);
    float acc[W];
#pragma unroll
    for (int i = 0; i < W; ++i) acc[i] = 0.0f;
    if (c < O) {
#pragma unroll 2
        for (int64_t t = t0 + threadIdx.y; t < t1; t += kSlopeRows) {
            const int64_t at = t * O + c;
            float v[W];
            if constexpr (W == 8) {
                const Words<4> gw = ld_stream<4>(g + at);
                Words<4> zw;
                if (act != kActNone) zw = ld_stream<4>(preact + at);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[2 * i] = Elem<DT>::lo(gw.w[i]), v[2 * i + 1] = Elem<DT>::hi(gw.w[i]);
                    if (act != kActNone) {
                        v[2 * i] *= slope(Elem<DT>::lo(zw.w[i]), act);
                        v[2 * i + 1] *= slope(Elem<DT>::hi(zw.w[i]), act);
                    }
                }
                if (u != nullptr) {
                    Words<4> o;
#pragma unroll
                    for (int i = 0; i < 4; ++i) o.w[i] = Elem<DT>::pack(v[2 * i], v[2 * i + 1]);
                    *reinterpret_cast<Words<4>*>(u + at) = o;
                }
            } else {
                v[0] = Elem<DT>::one(g[at]);
                if (act != kActNone) v[0] *= slope(Elem<DT>::one(preact[at]), act);
                if (u != nullptr) u[at] = Elem<DT>::cvt(v[0]);
            }
#pragma unroll
            for (int i = 0; i < W; ++i) acc[i] = __fadd_rn(acc[i], v[i]);
        }
    }
    if (partial == nullptr) return;
#pragma unroll
    for (int i = 0; i < W; ++i) part[threadIdx.y][threadIdx.x * W + i] = acc[i];
    __syncthreads();
    for (int i = threadIdx.y * 32 + threadIdx.x; i < 32 * W; i += 32 * kSlopeRows) {
        const int64_t o = int64_t(blockIdx.x) * 32 * W + i;
        if (o < O) {
            float s = part[0][i];
#pragma unroll
            for (int y = 1; y < kSlopeRows; ++y) s = __fadd_rn(s, part[y][i]);
            partial[int64_t(blockIdx.y) * O + o] = s;
        }
    }
}

}  // namespace linear
}  // namespace mhc
