// The kernels around the products of a cross entropy over a vocabulary
// (definitions in mhc_layer.h): the join of the groups' maxima and sums,
// the same and the logits' gradients from sums over runs of K, and the sum of
// grad_x's parts.
#pragma once

#include "mhc_linear.cuh"
#include "mhc_linear_plan.h"

namespace mhc {
namespace entropy {

// lse and loss from the units' pairs: THREADS threads a token (a warp, or a
// block where a token has more groups than kJoinGroups), thread i takes the groups i,
// i + THREADS, ... one after the other, a group's units in increasing order,
// then the threads' pairs meet in a tree; the order depends on V alone.
// Bound by the loads' latency where tokens are few (T = 8, V = 32768 6.1 us by
// itself, cold, about 3 behind the product), so four groups' are under way at a
// time (one: T = 200, 512 x 8000 9.7 us of the whole, four 7.7; T = 1, 2048 x 151936 104.7,
// 102.7), by HBM where they are many (T = 4096, V =
// 32768 13.3 us, cold).
constexpr int kJoinThreads = 256;
constexpr int kJoinGroups = 256;   // of a token that a warp joins; a block where there are more
constexpr int kJoinBatch = 4;   // groups of a thread whose loads are under way together

// Thread i's groups, of at most MOST units, and the threads' together (THREADS
// of them; part: shared memory for a pair a warp).
template <int THREADS, int MOST, typename Load>
__device__ __forceinline__ float2 join_units(Load load, int64_t units, uint32_t of_a_group, uint32_t i, float2* part) {
    float top = -INFINITY, sum = 0.0f;
    const int64_t step = int64_t(THREADS) * of_a_group;
    for (int64_t u0 = int64_t(i) * of_a_group; u0 < units; u0 += kJoinBatch * step) {
        float2 w[kJoinBatch][MOST];
#pragma unroll
        for (int j = 0; j < kJoinBatch; ++j)
#pragma unroll
            for (int k = 0; k < MOST; ++k)
                if (uint32_t(k) < of_a_group)
                    w[j][k] = u0 + j * step + k < units ? load(u0 + j * step + k) : make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int j = 0; j < kJoinBatch; ++j) {
            if (u0 + j * step >= units) break;
#pragma unroll
            for (int k = 1; k < MOST; ++k)
                if (uint32_t(k) < of_a_group) linear::join_groups(w[j][0].x, w[j][0].y, w[j][k].x, w[j][k].y);
            linear::join_groups(top, sum, w[j][0].x, w[j][0].y);
        }
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
        const float top2 = __shfl_xor_sync(0xFFFFFFFFu, top, s), sum2 = __shfl_xor_sync(0xFFFFFFFFu, sum, s);
        linear::join_groups(top, sum, top2, sum2);
    }
    if constexpr (THREADS > 32) {
        if (i % 32 == 0) part[i / 32] = make_float2(top, sum);
        umma::group_sync(1, THREADS);
        top = part[0].x, sum = part[0].y;
#pragma unroll
        for (int w = 1; w < THREADS / 32; ++w) linear::join_groups(top, sum, part[w].x, part[w].y);
    }
    return make_float2(top, sum);
}

template <int THREADS, int MOST>
static __global__ void __launch_bounds__(kJoinThreads)
join_kernel(const float2* __restrict__ partial, const float* __restrict__ at, const int64_t* __restrict__ target,
            float* __restrict__ loss, float* __restrict__ lse, int64_t T, int64_t V, int64_t units, uint32_t of_a_group) {
    pdl_enter();
    __shared__ float2 part[kJoinThreads / 32];
    const uint32_t i = threadIdx.x % THREADS;
    const int64_t t = int64_t(blockIdx.x) * (kJoinThreads / THREADS) + threadIdx.x / THREADS;
    const float2* p = partial + t * units;
    const float2 of = join_units<THREADS, MOST>([&](int64_t u) { return __ldcs(p + u); }, t < T ? units : 0, of_a_group, i, part);
    if (i == 0 && t < T) {
        const float all = __fadd_rn(linear::reference(of.x), logf(of.y));
        lse[t] = all;
        const int64_t entry = target[t];
        loss[t] = entry >= 0 && entry < V ? __fsub_rn(all, at[t]) : 0.0f;
    }
}

// lse and loss from the logits' sums over the runs of K, [runs,T,V], where
// those are tiles of their own: a block a token adds the runs up in increasing
// order, forms the units' pairs as few_kernel does and joins them as
// join_kernel does, so that the bits are theirs.  Bound by the loads' latency,
// so four entries a thread are under way at a time (one: T = 1, 7168 x 4096 21.4 us of
// the whole, four 18.8).
constexpr int kApartBatch = 4;   // entries of a thread whose loads are under way together
constexpr int kApartUnits = 2;   // of a group: so few entries are in groups of 32, at most as many as one warp joins in join_kernel
static_assert(linear::kApartEntries < linear::kWideGroups && linear::kApartEntries <= 32 * kJoinGroups);

template <int THREADS>
static __global__ void __launch_bounds__(THREADS)
apart_join_kernel(const float* __restrict__ sums, const int64_t* __restrict__ target, float* __restrict__ loss,
                  float* __restrict__ lse, int64_t T, int64_t V, uint32_t runs) {
    pdl_enter();
    extern __shared__ float2 pairs[];
    __shared__ float at;
    const int64_t t = blockIdx.x, units = (V + linear::kEntropyUnit - 1) / linear::kEntropyUnit;
    const int64_t entry = target[t];
    const float* p = sums + t * V;
    for (int64_t n0 = threadIdx.x; n0 - threadIdx.x % 32 < V; n0 += kApartBatch * THREADS) {
        float x[kApartBatch];
#pragma unroll
        for (int k = 0; k < kApartBatch; ++k) x[k] = n0 + k * THREADS < V ? __ldcs(p + n0 + k * THREADS) : -INFINITY;
#pragma unroll 4
        for (uint32_t r = 1; r < runs; ++r) {
            const float* q = p + int64_t(r) * T * V + n0;
#pragma unroll
            for (int k = 0; k < kApartBatch; ++k)
                if (n0 + k * THREADS < V) x[k] = __fadd_rn(x[k], __ldcs(q + k * THREADS));
        }
#pragma unroll
        for (int k = 0; k < kApartBatch; ++k) {
            const int64_t n = n0 + k * THREADS;
            if (n - threadIdx.x % 32 >= V) break;   // (the same for the whole warp)
            if (n == entry) at = x[k];
            const float2 of = linear::entropy_unit(x[k]);
            if (threadIdx.x % linear::kEntropyUnit == 0 && n < V) pairs[n / linear::kEntropyUnit] = of;
        }
    }
    __syncthreads();
    if (threadIdx.x >= 32) return;
    const float2 of = join_units<32, kApartUnits>([&](int64_t u) { return pairs[u]; }, units, kApartUnits, threadIdx.x, nullptr);
    if (threadIdx.x == 0) {
        const float all = __fadd_rn(linear::reference(of.x), logf(of.y));
        lse[t] = all;
        loss[t] = entry >= 0 && entry < V ? __fsub_rn(all, at) : 0.0f;
    }
}

// The logits' gradients (as kEndProb's) from such sums: two entries of a token
// a thread.
constexpr int kApartGradThreads = 256;

template <int DT>
static __global__ void __launch_bounds__(kApartGradThreads)
apart_grad_kernel(const float* __restrict__ sums, const linear::TileArgs a, int64_t V, uint32_t runs, uint32_t by_token) {
    pdl_enter();
    const linear::Scale scale = linear::scale_of<kApartGradThreads>(a.end, a.rows);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.end.inverse = scale.inverse;
    const int64_t t = blockIdx.x / by_token, n = (int64_t(blockIdx.x % by_token) * kApartGradThreads + threadIdx.x) * 2;
    if (n >= V) return;
    const linear::RowHead h = linear::row_head<linear::kEndProb>(a, t, true, scale.by);
    const bool two = n + 1 < V;
    const float* p = sums + t * V + n;
    float x = __ldcs(p), y = two ? __ldcs(p + 1) : 0.0f;
#pragma unroll 4
    for (uint32_t r = 1; r < runs; ++r) {
        const float* q = p + int64_t(r) * a.rows * V;
        x = __fadd_rn(x, __ldcs(q));
        if (two) y = __fadd_rn(y, __ldcs(q + 1));
    }
    const bool some = h.factor != 0.0f;
    x = some ? __fmul_rn(linear::exp_fast(__fsub_rn(x, h.lse)), h.factor) : 0.0f;
    y = some ? __fmul_rn(linear::exp_fast(__fsub_rn(y, h.lse)), h.factor) : 0.0f;
    if (h.at == n) x = __fsub_rn(x, h.target_grad);
    if (h.at == n + 1) y = __fsub_rn(y, h.target_grad);
    *reinterpret_cast<uint32_t*>(a.e.y + t * a.end.pitch + n) = Elem<DT>::pack(x, y);   // (the pitch is even and holds the pair)
}

// A gradient from its parts' sums: their sum in increasing order, scaled (where scale is not null) and rounded.
constexpr int kSumThreads = 256;

template <int DT>
static __global__ void __launch_bounds__(kSumThreads)
sum_kernel(const float* __restrict__ sums, const float* __restrict__ scale, uint16_t* __restrict__ out, int64_t n, uint32_t parts) {
    pdl_enter();
    const float f = scale == nullptr ? 1.0f : *scale;
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

}  // namespace entropy
}  // namespace mhc
