// The kernels around the products of a cross entropy over a vocabulary
// (definitions in mhc_layer.h): the join of the groups' maxima and sums, and
// what each token brings to the gradient of its logits.
#pragma once

#include "mhc_linear.cuh"

namespace mhc {
namespace entropy {

// lse and loss from the units' pairs: THREADS threads a token (a warp, or a
// block where a token has more groups than 256), thread i takes the groups i,
// i + THREADS, ... one after the other, a group's units in increasing order,
// then the threads' pairs meet in a tree; the order depends on V alone.
// Bound by the loads' latency: T = 8, V = 32768 FIG_JOIN us.
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
sum_kernel(const float* __restrict__ sums, const float* __restrict__ factor, uint16_t* __restrict__ out, int64_t n, uint32_t parts) {
    pdl_enter();
    const float f = *factor;
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

// Each token's part of d, times a power of two that brings the largest
// gradient to 2^13 .. 2^14: binary16 operands then hold probabilities down to
// 2^-38 of it (BF16 ones need it not and lose nothing).  factor: its inverse.
// One block, since the power is of all tokens.
constexpr int kTokenThreads = 1024;

static __global__ void __launch_bounds__(kTokenThreads)
token_kernel(const float* __restrict__ grad_loss, const float* __restrict__ grad_lse, const int64_t* __restrict__ target,
             const float* __restrict__ lse, linear::EntropyToken* __restrict__ tokens, float* __restrict__ factor, int64_t T,
             int64_t V) {
    pdl_enter();
    __shared__ float most[kTokenThreads / 32];
    auto gradients = [&](int64_t t, float& spread, float& at_target, int64_t& entry) {
        entry = target[t];
        at_target = grad_loss != nullptr && entry >= 0 && entry < V ? grad_loss[t] : 0.0f;
        spread = grad_lse == nullptr ? at_target : __fadd_rn(at_target, grad_lse[t]);
    };
    float m = 0.0f;
    for (int64_t t = threadIdx.x; t < T; t += kTokenThreads) {
        float spread, at_target;
        int64_t entry;
        gradients(t, spread, at_target, entry);
        m = fmaxf(m, fmaxf(fabsf(spread), fabsf(at_target)));
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
    if (threadIdx.x % 32 == 0) most[threadIdx.x / 32] = m;
    __syncthreads();
    m = most[threadIdx.x % 32];
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
    int power = 0;
    if (m > 0.0f && m < INFINITY) power = min(13 - ilogbf(m), 126);
    const float scale = ldexpf(1.0f, power);
    if (threadIdx.x == 0) *factor = ldexpf(1.0f, -power);
    for (int64_t t = threadIdx.x; t < T; t += kTokenThreads) {
        float spread, at_target;
        int64_t entry;
        gradients(t, spread, at_target, entry);
        linear::EntropyToken k;
        k.lse = lse[t];
        k.spread = __fmul_rn(spread, scale);
        k.target_grad = __fmul_rn(at_target, scale);
        k.target = entry >= 0 && entry < V ? int32_t(entry) : -1;
        tokens[t] = k;
    }
}

}  // namespace entropy
}  // namespace mhc
