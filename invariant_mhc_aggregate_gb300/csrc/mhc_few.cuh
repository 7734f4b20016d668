// Products of few rows (sm_103a): the weight's bytes are the whole cost, so
// its rows are dealt out evenly to all SMs and stream without a pause.
#pragma once

#include "mhc_linear.cuh"

namespace mhc {
namespace linear {

// One persistent CTA an SM takes tiles of a.lanes output columns (weight rows,
// a multiple of 16, at most 128: as many as make the CTAs' shares even) by all
// of the call's rows, at most WIDTH.  Against split_kernel, whose tiles are
// always 128 lanes and end in an epilogue of their own, no SM has a tile more
// than the others and the copies of the next tile run under the end of this
// one: T = 1, 8-bit 7168 -> 2 x 14336 36.1 -> 33.6 us (6.1 TB/s), T = 64 38.3
// -> 36.7.  A cross entropy of few tokens leaves pair_kernel's tiles of 256
// tokens for it: T = 8, I = 2048, 32768 entries 34.9 -> 26.9 us with the join,
// T = 64 32.4 -> 29.6.  Rows past 64 would not gain (T = 128, 7168 -> 2 x 14336
// 71.5 us in the other kernels, 75.4 in this one).
//
// The multiplications are 128 lanes high whatever a.lanes is: the rows of
// shared memory past them are never written, and what they bring stays in
// lanes that nobody reads.
//
// Parts of K are summed apart, in kSlots accumulators in turn, and added in
// increasing order in registers: the bits of split_kernel and pair_kernel.
//
// Warps 0 .. 4 groups - 1 read tensor memory (a group is four warps, for the
// quarters of the lanes, and has 8 or 16 columns), then one warp copies and one
// multiplies.
constexpr uint32_t kSlots = 4;

template <int WIDTH>
constexpr int kFewGroups = WIDTH < 32 ? WIDTH / 8 : 4;
template <int WIDTH>
constexpr uint32_t kFewThreads = 32 * (4 * kFewGroups<WIDTH> + 2);

// Blocks of K of a CTA's first tile that go to L2 before the launch's wait.
constexpr uint32_t kAhead = 8;

// load_p's boxes into L2.
template <bool FP8, int END>
__device__ __forceinline__ void prefetch_p(const CUtensorMap* mp, uint32_t k, int p0, int half) {
    const int k0 = int(k * (FP8 ? 128u : 64u));
    umma::tensor_prefetch_2d(mp, k0, END == kEndGated ? p0 / 2 : p0);
    if constexpr (END == kEndGated) umma::tensor_prefetch_2d(mp, k0, half + p0 / 2);
}

// The groups' maxima and sums of one tile: 16 lanes are 16 entries of the
// vocabulary, and v one token's logit of each (entropy_tile has the same sums
// in the same order).
template <int C>
__device__ __forceinline__ void entropy_lanes(const TileArgs& a, uint32_t m0, int64_t n, bool n_ok, float (&v)[C]) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const uint32_t m = m0 + c;
        if (m >= a.rows) break;   // (the same for the whole warp)
        if (n_ok && __ldg(a.end.target + m) == n) a.end.at[m] = v[c];
        const float2 of = entropy_unit(n_ok ? v[c] : -INFINITY);
        if ((threadIdx.x & 15) == 0 && n_ok) a.end.partial[int64_t(m) * a.end.units + n / kEntropyUnit] = of;
    }
}

template <bool FP8, int OUT, int WIDTH, int END>
__global__ void __launch_bounds__(kFewThreads<WIDTH>, 1)
few_kernel(const __grid_constant__ CUtensorMap mp, const __grid_constant__ CUtensorMap mq, const __grid_constant__ TileArgs a) {
    constexpr int kGroups = kFewGroups<WIDTH>, C = WIDTH / kGroups;   // columns of a thread
    constexpr uint32_t kReaders = 4 * kGroups, kColumns = kSlots * WIDTH;
    extern __shared__ char raw[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], sum_full[kSlots], sum_empty[kSlots];
    __shared__ uint32_t tmem_base;
    char* stages = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // (with kEndSum the parts of K are tiles of their own, as in pair_kernel)
    constexpr bool kApart = END == kEndSum;
    const uint32_t tiles = kApart ? a.p_tiles * a.splits : a.p_tiles;
    auto tile_of = [&](uint32_t i) { return kApart ? i % a.p_tiles : i; };
    auto first_part = [&](uint32_t i) { return kApart ? i / a.p_tiles : 0u; };
    auto last_part = [&](uint32_t i) { return kApart ? i / a.p_tiles + 1 : a.splits; };
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < a.stages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (uint32_t s = 0; s < kSlots; ++s) {
            mbar_init(sum_full + s, 1);
            mbar_init(sum_empty + s, kReaders);
        }
        mbar_init_fence();
    }
    if (warp == kReaders) {
        umma::tmem_alloc<1>(&tmem_base, kColumns);
        umma::tmem_relinquish<1>();
        if (lane == 0) {
            umma::prefetch_map(&mp);
            umma::prefetch_map(&mq);
        }
    }
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = tmem_base;
    // The tile's first blocks of the weight go to L2 while the launch before still
    // runs: what that writes is in L2 too, so a weight of its making is copied as
    // it left it.  T = 1, 2048 -> 2 x 8192 13.0 -> 12.4 us, T = 8, 2048 x 32768 26.6 -> 26.3;
    // 24 blocks 11.8 and 26.0, but T = 16, 2048 -> 2 x 10240 17.0 -> 18.4.
    if (warp == kReaders + 1 && blockIdx.x < tiles && umma::elect()) {
        const uint32_t part = first_part(blockIdx.x), k0 = split_begin(a, part);
        const uint32_t k1 = min(kApart ? split_begin(a, part + 1) : a.kb, k0 + kAhead);
        for (uint32_t k = k0; k < k1; ++k) prefetch_p<FP8, END>(&mp, k, int(tile_of(blockIdx.x) * a.lanes), int(a.end.half));
    }
    __syncwarp();
    pdl_enter();
    const uint32_t ring = smem_addr(stages), bar_full = smem_addr(full), bar_empty = smem_addr(empty);
    const uint32_t bar_sum = smem_addr(sum_full), bar_free = smem_addr(sum_empty);
    const uint32_t count = a.stages, bytes = a.stage_bytes, unit = a.unit;
    if (warp == kReaders) {
        umma::Ring at;
        bool ok = true;
        uint32_t issued = 0;
        for (uint32_t i = blockIdx.x; i < tiles && ok; i += gridDim.x) {
            const int p0 = int(tile_of(i) * a.lanes);
            uint32_t k = kApart ? split_begin(a, first_part(i)) : 0;
            for (uint32_t part = first_part(i); part < last_part(i) && ok; ++part) {
                for (const uint32_t k1 = split_begin(a, part + 1); k < k1; ++issued, at.next(count)) {
                    if (!(ok = umma::wait_warp(bar_empty + 8 * at.stage, at.parity ^ 1))) break;
                    const uint32_t n = min(unit, k1 - k);
                    if (umma::elect()) {
                        umma::expect_tx(bar_full + 8 * at.stage, n * (a.lanes + WIDTH) * 128);
                        for (uint32_t u = 0; u < n; ++u) {
                            const uint32_t to = ring + at.stage * bytes + u * a.block_bytes;
                            load_p<1, FP8, kBothK, END>(to, &mp, k + u, p0, bar_full + 8 * at.stage, int(a.end.half), a.lanes);
                            load_q<1, FP8, kBothK>(to, &mq, k + u, 0, WIDTH, bar_full + 8 * at.stage);
                        }
                    }
                    __syncwarp();
                    k += n;
                }
            }
        }
        drain(ok, min(issued, count), at, count, bar_empty, bar_full);
        if (!ok) timed_out(a);
    } else if (warp == kReaders + 1) {
        const Descs d = descs<kBothK>(ring);
        const uint32_t idesc = a.idesc;
        umma::Ring at, sums;
        bool ok = true;
        for (uint32_t i = blockIdx.x; i < tiles && ok; i += gridDim.x) {
            uint32_t k = kApart ? split_begin(a, first_part(i)) : 0;
            for (uint32_t part = first_part(i); part < last_part(i) && ok; ++part, sums.next(kSlots)) {
                if (!(ok = umma::wait_warp(bar_free + 8 * sums.stage, sums.parity ^ 1))) break;
                umma::fence_after_sync();
                const uint32_t to = tmem + sums.stage * WIDTH, k0 = k, k1 = split_begin(a, part + 1);
                for (; k < k1; at.next(count)) {
                    if (!(ok = umma::wait_warp(bar_full + 8 * at.stage, at.parity))) break;
                    umma::fence_after_sync();
                    const uint32_t n = min(unit, k1 - k);
                    if (umma::elect()) {
                        for (uint32_t u = 0; u < n; ++u)
                            multiply_block<1, FP8, kBothK>(d, at.stage * bytes + u * a.block_bytes, idesc, to, k + u == k0);
                        umma::commit<1>(bar_empty + 8 * at.stage);
                        if (k + n == k1) umma::commit<1>(bar_sum + 8 * sums.stage);
                    }
                    __syncwarp();
                    k += n;
                }
            }
        }
        if (!ok) timed_out(a);
    } else {
        const uint32_t quarter = warp % 4, m0 = warp / 4 * C;   // the thread's lane, its columns m0 .. m0 + C
        const uint32_t in_tile = quarter * 32 + lane;
        const uint32_t tw = tmem + (quarter * 32u << 16) + m0;
        constexpr bool kTogether = END == kEndGated;   // (as in pair_kernel)
        umma::Ring sums;
        bool ok = true;
        for (uint32_t i = blockIdx.x; i < tiles && (ok || kTogether); i += gridDim.x) {
            int64_t n = int64_t(tile_of(i)) * a.lanes + in_tile;
            bool n_ok = n < a.N && in_tile < a.lanes;
            Gated gated;
            if constexpr (END == kEndGated) gated = gated_place(a, stages, warp / 4, in_tile, int64_t(i) * (a.lanes / 2), n, n_ok);
            const float bias = a.e.bias != nullptr && n_ok ? __ldg(a.e.bias + n) : 0.0f;
            const float cs = a.e.col_scale != nullptr && n_ok ? __ldg(a.e.col_scale + n) : 1.0f;
            float v[C / 8][8];
            for (uint32_t part = first_part(i); part < last_part(i); ++part, sums.next(kSlots)) {
                ok = ok && umma::wait_warp(bar_sum + 8 * sums.stage, sums.parity);
                if (!ok && !kTogether) break;
                umma::fence_after_sync();
                const uint32_t from = tw + sums.stage * WIDTH;
                if (kApart || part == 0) {
#pragma unroll
                    for (int c = 0; c < C / 8; ++c) umma::tmem_ld(from + 8 * c, v[c]);
#pragma unroll
                    for (int c = 0; c < C / 8; ++c) umma::tmem_wait_ld(v[c]);
                } else {
                    float w[C / 8][8];
#pragma unroll
                    for (int c = 0; c < C / 8; ++c) umma::tmem_ld(from + 8 * c, w[c]);
#pragma unroll
                    for (int c = 0; c < C / 8; ++c) {
                        umma::tmem_wait_ld(w[c]);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[c][j] = __fadd_rn(v[c][j], w[c][j]);
                    }
                }
                umma::fence_before_sync();
                __syncwarp();
                if (lane == 0) umma::arrive_cluster(bar_free + 8 * sums.stage);
            }
            if (!ok && !kTogether) break;
#pragma unroll
            for (int c = 0; c < C / 8; ++c) {
                if (m0 + 8 * c >= a.rows) break;
                if constexpr (END == kEndEntropy) entropy_lanes<8>(a, m0 + 8 * c, n, n_ok, v[c]);
                else if constexpr (END == kEndSum) emit_sum<OUT, 8, false>(a, n_ok, n, m0 + 8 * c, 1, a.rows, v[c], first_part(i));
                else gated_chunk<OUT>(a, gated, n_ok, n, m0 + 8 * c, 1, a.rows, v[c], bias, cs);
            }
        }
        if (!ok) timed_out(a);
        umma::fence_before_sync();
    }
    __syncthreads();
    umma::fence_after_sync();
    if (warp == kReaders) umma::tmem_free<1>(tmem, kColumns);
}

}  // namespace linear
}  // namespace mhc
