// The kernels around the products of a cross entropy over a vocabulary
// (definitions in mhc_layer.h): the join of the groups' maxima and sums,
// the sum of grad_x's parts, and the scale of binary16 gradients.
#pragma once

#include "mhc_linear.cuh"

namespace mhc {
namespace entropy {

// lse and loss from the units' pairs: THREADS threads a token (a warp, or a
// block where a token has more groups than 256), thread i takes the groups i,
// i + THREADS, ... one after the other, a group's units in increasing order,
// then the threads' pairs meet in a tree; the order depends on V alone.
// Bound by the loads' latency where tokens are few (T = 8, V = 32768 6.1 us by
// itself, about 3 behind the product), by HBM where they are many (T = 4096, V =
// 32768 13.3 us, cold).
constexpr int kJoinThreads = 256;

template <int THREADS>
static __global__ void __launch_bounds__(kJoinThreads)
join_kernel(const float2* __restrict__ partial, const float* __restrict__ at, const int64_t* __restrict__ target,
            float* __restrict__ loss, float* __restrict__ lse, int64_t T, int64_t V, int64_t units, uint32_t of_a_group) {
    pdl_enter();
    const uint32_t i = threadIdx.x % THREADS;
    const int64_t t = int64_t(blockIdx.x) * (kJoinThreads / THREADS) + threadIdx.x / THREADS;
    float top = -INFINITY, sum = 0.0f;
    if (t < T) {
        const float2* p = partial + t * units;
        for (int64_t u = int64_t(i) * of_a_group; u < units; u += int64_t(THREADS) * of_a_group) {
            float2 w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (uint32_t(k) < of_a_group) w[k] = u + k < units ? __ldcs(p + u + k) : make_float2(-INFINITY, 0.0f);
#pragma unroll
            for (int k = 1; k < 4; ++k)
                if (uint32_t(k) < of_a_group) linear::join_groups(w[0].x, w[0].y, w[k].x, w[k].y);
            linear::join_groups(top, sum, w[0].x, w[0].y);
        }
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
        const float top2 = __shfl_xor_sync(0xFFFFFFFFu, top, s), sum2 = __shfl_xor_sync(0xFFFFFFFFu, sum, s);
        linear::join_groups(top, sum, top2, sum2);
    }
    if constexpr (THREADS > 32) {
        __shared__ float2 part[THREADS / 32];
        if (i % 32 == 0) part[i / 32] = make_float2(top, sum);
        __syncthreads();
        top = part[0].x, sum = part[0].y;
#pragma unroll
        for (int w = 1; w < THREADS / 32; ++w) linear::join_groups(top, sum, part[w].x, part[w].y);
    }
    if (i == 0 && t < T) {
        const float all = __fadd_rn(linear::reference(top), logf(sum));
        lse[t] = all;
        const int64_t entry = target[t];
        loss[t] = entry >= 0 && entry < V ? __fsub_rn(all, at[t]) : 0.0f;
    }
}

// grad_x from the parts' sums: their sum in increasing order, scaled and rounded.
constexpr int kSumThreads = 256;

template <int DT>
static __global__ void __launch_bounds__(kSumThreads)
sum_kernel(const float* __restrict__ sums, const float* __restrict__ scale, uint16_t* __restrict__ out, int64_t n, uint32_t parts) {
    pdl_enter();
    const float f = scale == nullptr ? 1.0f : scale[1];
    const int64_t i = (int64_t(blockIdx.x) * kSumThreads + threadIdx.x) * 2;
    if (i >= n) return;
    const bool two = i + 1 < n;
    float a = 0.0f, b = 0.0f;
#pragma unroll 4
    for (uint32_t p = 0; p < parts; ++p) {
        const float* q = sums + int64_t(p) * n + i;
        const float x = __ldcs(q), y = two ? __ldcs(q + 1) : 0.0f;
        a = p == 0 ? x : __fadd_rn(a, x);
        b = p == 0 ? y : __fadd_rn(b, y);
    }
    out[i] = Elem<DT>::cvt(__fmul_rn(a, f));
    if (two) out[i + 1] = Elem<DT>::cvt(__fmul_rn(b, f));
}

// Binary16 alone: scale[0] is a power of two that brings the largest gradient
// of a token to 2^13 .. 2^14, so that the logits' gradients hold probabilities
// down to 2^-38 of it, and scale[1] its inverse.  One block, since it is of all
// tokens.
constexpr int kScaleThreads = 1024;

static __global__ void __launch_bounds__(kScaleThreads)
scale_kernel(const float* __restrict__ grad_loss, const float* __restrict__ grad_lse, const int64_t* __restrict__ target,
             float* __restrict__ scale, int64_t T, int64_t V) {
    pdl_enter();
    __shared__ float most[kScaleThreads / 32];
    float m = 0.0f;
    for (int64_t t = threadIdx.x; t < T; t += kScaleThreads) {
        const int64_t entry = target[t];
        const float g = grad_loss != nullptr && entry >= 0 && entry < V ? grad_loss[t] : 0.0f;
        const float spread = grad_lse == nullptr ? g : __fadd_rn(g, grad_lse[t]);
        m = fmaxf(m, fmaxf(fabsf(spread), fabsf(g)));
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
    if (threadIdx.x % 32 == 0) most[threadIdx.x / 32] = m;
    __syncthreads();
    if (threadIdx.x >= 32) return;
    m = most[threadIdx.x];
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
    if (threadIdx.x != 0) return;
    int power = 0;
    if (m > 0.0f && m < INFINITY) power = min(13 - ilogbf(m), 126);
    scale[0] = ldexpf(1.0f, power);
    scale[1] = ldexpf(1.0f, -power);
}

}  // namespace entropy
}  // namespace mhc
