// The kernels around the products of a cross entropy over a vocabulary
// (definitions in mhc_layer.h): the join of the groups' maxima and sums, and
// what each token brings to the gradient of its logits.
#pragma once

#include "mhc_linear.cuh"

namespace mhc {
namespace entropy {

// lse and loss of 32 tokens a block: worker i takes the groups i, i + 32, ...
// one after the other, then the workers' pairs meet in a tree; the order
// depends on the number of groups alone.  HBM-bound where tokens are many
// (8 bytes a group and token), by the loads' latency where they are few.
constexpr int kWorkers = 32;

static __global__ void __launch_bounds__(32 * kWorkers)
join_kernel(const float2* __restrict__ partial, const float* __restrict__ at, const int64_t* __restrict__ target,
            float* __restrict__ loss, float* __restrict__ lse, int64_t T, int64_t V, uint32_t groups) {
    pdl_enter();
    const uint32_t lane = threadIdx.x % 32, worker = threadIdx.x / 32;
    __shared__ float2 part[kWorkers][32];
    const int64_t t = int64_t(blockIdx.x) * 32 + lane;
    float top = -INFINITY, sum = 0.0f;
    if (t < T) {
        const float2* p = partial + t;
        uint32_t g = worker;
        constexpr int kAhead = 4;
        for (; g + (kAhead - 1) * kWorkers < groups; g += kAhead * kWorkers) {
            float2 w[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) w[i] = __ldcs(p + int64_t(g + i * kWorkers) * T);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) linear::join_groups(top, sum, w[i].x, w[i].y);
        }
        for (; g < groups; g += kWorkers) {
            const float2 w = __ldcs(p + int64_t(g) * T);
            linear::join_groups(top, sum, w.x, w.y);
        }
    }
    part[worker][lane] = make_float2(top, sum);
    for (int s = kWorkers / 2; s > 0; s >>= 1) {
        __syncthreads();
        if (int(worker) < s) {
            const float2 w = part[worker + s][lane];
            linear::join_groups(top, sum, w.x, w.y);
            part[worker][lane] = make_float2(top, sum);
        }
    }
    if (worker == 0 && t < T) {
        const float all = __fadd_rn(linear::reference(top), logf(sum));
        lse[t] = all;
        const int64_t at_entry = target[t];
        loss[t] = at_entry >= 0 && at_entry < V ? __fsub_rn(all, at[t]) : 0.0f;
    }
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
