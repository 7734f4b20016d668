// Which kernel a matrix product takes, with which tiles and parts of K
// (mhc_linear.cuh).  The plan fixes the order of the product's sums, so it
// follows from the sizes alone: GB300's counts are constants here, no device
// is asked, and every device and process gives the same bits.
#pragma once

#include <stdint.h>

namespace mhc {
namespace linear {

// Clusters of 1, 2, 4 and 8 CTAs (one an SM) that GB300 runs at once: its
// SMs come in groups that a cluster does not cross.
constexpr int64_t kClustersAtOnce[4] = {152, 76, 36, 15};
constexpr int64_t kPairsAtOnce = kClustersAtOnce[1];   // of pair_kernel's CTAs

// Parts of K: as many (1, 2, 4 or 8) as run at once when the call has `tiles`
// tiles of 128 lanes, with at least 8 blocks of K a part.  Joining parts takes
// about 1.9 us, as long as 10 blocks: fewer than 24 blocks stay in one part.
// Returns the logarithm.
inline uint32_t splits_of(int64_t tiles, int64_t kb) {
    uint32_t s = 0;
    if (kb < 24) return s;
    while (s < 3 && tiles <= kClustersAtOnce[s + 1] && kb >= (16 << s)) ++s;
    return s;
}

// Which kernel a product takes, with tiles of which width (output rows).
struct Plan {
    bool pair;
    uint32_t width, splits;
};

// The cheapest plan by an estimate in SM cycles, fitted to runs of M = 16 ..
// 2048 rows at (N, K) = (7168, 7168), (14336, 4096), (4096, 4096), (4096, 1280),
// (2048, 2048), (1024, 1024), (1024, 7168), (520, 2048), (640, 512):
//  * split_kernel: each round of the clusters that run at once takes 4500 + 24
//    width for its start and epilogue, 3600 to join parts, and 260 + width a
//    block of K;
//  * pair_kernel: 6000 + 21 width once, each round max(300, 2.05 width) a block
//    of K and 1500 a part.
// For instance M = 256 at 4096 x 4096: split 16.0 us, pairs 20.2; M = 512: 31.1
// and 20.8; M = 1024 at 1024 x 1024: split 6.2 us in tiles of 64 rows, 10.1 in
// tiles of 256, pairs 7.3; M = 2048 at 7168 x 7168: pairs of width 256 115.7 us,
// 128 138.8, split 188.
inline Plan plan_of(int64_t N, int64_t M, int64_t kb, bool q_mn, bool by_row) {
    const int64_t p128 = (N + 127) / 128, p256 = (N + 255) / 256;
    Plan best = {false, 256, 1};
    int64_t least = INT64_MAX;
    // where a row's sum must not depend on how many rows the call has, the parts
    // follow from N and K alone: those of a call with few rows
    const uint32_t row_log = splits_of(p128, kb);
    const int64_t step = q_mn ? 64 : 16, q0 = (M + 255) / 256;
    for (int64_t q = q0; q <= 8 * q0 && q <= 65535; q *= 2) {   // (its grid's second dimension)
        const int64_t w = ((M + q - 1) / q + step - 1) / step * step;
        const int64_t tiles = p128 * ((M + w - 1) / w);
        const uint32_t log = by_row ? row_log : splits_of(tiles, kb), parts = 1u << log;
        const int64_t rounds = (tiles + kClustersAtOnce[log] - 1) / kClustersAtOnce[log];
        const int64_t cost = rounds * (4500 + 24 * w + (parts > 1 ? 3600 : 0) + (kb + parts - 1) / parts * (260 + w));
        if (cost < least) least = cost, best = {false, uint32_t(w), parts};
        if (w <= 32) break;
    }
    const uint32_t parts = by_row ? 1u << row_log : 1;
    for (int64_t w = 128; w <= 256; w += q_mn ? 128 : 32) {
        const int64_t rounds = (p256 * ((M + w - 1) / w) + kPairsAtOnce - 1) / kPairsAtOnce;
        const int64_t block = 41 * w / 20 > 300 ? 41 * w / 20 : 300;
        const int64_t cost = 6000 + 21 * w + rounds * (kb * block + (parts > 1 ? 1500 * parts : 0));
        if (cost < least) least = cost, best = {true, uint32_t(w), parts};
    }
    return best;
}

// few_kernel: rows it takes, its tiles' columns of them, and the lanes (weight
// rows) that make the SMs' shares even: as few rounds of tiles as 128 lanes
// allow, each of them full.
constexpr int64_t kFewRows = 64;

inline uint32_t few_width(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : 64; }

inline uint32_t few_lanes(int64_t N) {
    const int64_t sms = kClustersAtOnce[0], rounds = (N + 128 * sms - 1) / (128 * sms);
    const int64_t lanes = ((N + sms * rounds - 1) / (sms * rounds) + 15) / 16 * 16;
    return uint32_t(lanes < 128 ? lanes : 128);
}

// A cross entropy's logits are summed in runs of at most 16 blocks of K
// (mhc_linear_ends.cuh says why).  A small vocabulary has few tiles, each of
// which goes through all of K by itself: there the runs are tiles of their
// own, whose sums meet in memory, in FP32, in the same order (I = 7168 and V = 1024:
// T = 1 26.3 -> 9.6 us, T = 128 27.5 -> 11.7, T = 512 27.6 -> 18.0; I = 2048, V = 4096: T = 16
// 13.2 -> 9.9).  Past these limits the sums' way costs more than the empty SMs
// (V = 12288: T = 1, I = 7168 32.4 us, so 45.8; T = 256, 4096 x 4096 19.5, so 28.5); at
// them the two are even (V = 8192: T = 1, I = 4096 20.1, 20.3; T = 64 25.0, 20.9).
constexpr uint32_t kEntropyRun = 16;

// Entries of the vocabulary that are summed together before the join: they
// follow from V alone, so that a token's loss has the same bits in every
// batch: 64, and 32 where tiles of 64 a thread would leave SMs without one.
// With few tokens few_kernel writes their units of 16.
constexpr int64_t kWideGroups = 256 * kPairsAtOnce;   // the smallest vocabulary with 64

inline int64_t entropy_group(int64_t V) { return V >= kWideGroups ? 64 : 32; }

constexpr int64_t kApartEntries = 8192;   // the largest vocabulary whose runs are tiles of their own

inline uint32_t entropy_runs(int64_t kb) { return uint32_t((kb + kEntropyRun - 1) / kEntropyRun); }

inline bool entropy_apart(int64_t T, int64_t V, int64_t kb) {
    return kb > kEntropyRun && V <= kApartEntries && T <= 512 && T * V <= int64_t(1) << 19;
}

// few_kernel's lanes for such tiles, and pair_kernel's width (of tokens): the cheapest
// rounds of `runs` tiles for each of theirs.  A block of K costs few_kernel its
// multiplications or its copies (24 bytes a cycle and SM).
inline uint32_t apart_lanes(int64_t N, int64_t runs) {
    uint32_t best = 128;
    int64_t least = INT64_MAX;
    for (int64_t lanes = 128; lanes >= 16; lanes -= 16) {
        const int64_t rounds = ((N + lanes - 1) / lanes * runs + kClustersAtOnce[0] - 1) / kClustersAtOnce[0];
        const int64_t cost = rounds * (280 > 16 * lanes / 3 ? 280 : 16 * lanes / 3);
        if (cost < least) least = cost, best = uint32_t(lanes);
    }
    return best;
}

inline uint32_t apart_width(int64_t N, int64_t M, int64_t runs) {
    uint32_t best = 128;
    int64_t least = INT64_MAX;
    for (int64_t w = 128; w <= 256; w += 32) {
        const int64_t rounds = ((N + 255) / 256 * ((M + w - 1) / w) * runs + kPairsAtOnce - 1) / kPairsAtOnce;
        const int64_t cost = 21 * w + rounds * (kEntropyRun * (41 * w / 20 > 300 ? 41 * w / 20 : 300) + 1500);
        if (cost < least) least = cost, best = uint32_t(w);
    }
    return best;
}

// Entries of the vocabulary whose logits' gradients are in the workspace at a
// time: 19456 (a tile of 256 for each pair of CTAs), more with fewer tokens
// (256 MB: T = 1024, 1024 x 128000 591 us in pieces of 32 MB, 497; T = 4096, 7168 x
// 131072 13.8 ms in pieces of 160 MB, 13.3), fewer with very many (1 GB).
inline int64_t entropy_piece(int64_t T, int64_t V) {
    int64_t n = 256 * kPairsAtOnce;
    if (T * n < int64_t(1) << 27) n = (int64_t(1) << 27) / T;
    if (T * n > int64_t(1) << 29) n = (int64_t(1) << 29) / T;
    if (n < 4096) n = 4096;
    const int64_t pieces = (V + n - 1) / n;
    return ((V + pieces - 1) / pieces + 63) / 64 * 64;
}

// The most blocks of K that one accumulator sums where K is tokens or a
// vocabulary (16384 of them): the tensor cores cut off each addition's last
// bits, so that a sum of terms of one sign falls short by a part that grows with
// them (65536 tokens in one accumulator 1.7e-4, 1048576 6.5e-3, in runs of this
// length 1.4e-5 both).  The runs are added up in FP32, rounded to nearest.
constexpr int64_t kSumBlocks = 256;

inline uint32_t sum_parts(int64_t kb) { return uint32_t((kb + kSumBlocks - 1) / kSumBlocks); }

// A gradient summed over `kb` blocks of K, [M,N]: pairs of CTAs, tiles of `width`
// rows (a multiple of `step`), and parts of K that are tiles of their own, so
// that few tiles fill the GPU.  The cheapest by plan_of's estimate of a round;
// joining parts costs their sums' way through memory.
inline Plan sum_plan(int64_t N, int64_t M, int64_t kb, int64_t step = 32) {
    Plan best = {true, 128, 1};
    int64_t least = INT64_MAX;
    for (int64_t parts = sum_parts(kb); parts == sum_parts(kb) || (parts <= 32 && kb >= 4 * parts); ++parts) {
        const int64_t join = parts > 1 ? 4000 + parts * M * N * 8 / 3000 : 0, blocks = (kb + parts - 1) / parts;
        for (int64_t w = 128; w <= 256; w += step) {
            const int64_t rounds = ((N + 255) / 256 * ((M + w - 1) / w) * parts + kPairsAtOnce - 1) / kPairsAtOnce;
            const int64_t block = 41 * w / 20 > 300 ? 41 * w / 20 : 300;
            const int64_t cost = 6000 + 21 * w + rounds * (blocks * block + 1500) + join;
            if (cost < least) least = cost, best = {true, uint32_t(w), uint32_t(parts)};
        }
    }
    return best;
}

// A gated product's grad_w [M,N] over `kb` blocks of tokens: the product's plan,
// with pair_kernel's tiles summed in parts one after the other.  Few tiles go to
// split_kernel, whose parts are a cluster's CTAs; where there are more tokens than
// those sum (token_apart), the parts are tiles of their own (sum_plan).  Whole
// backward, long runs and these: T = 65536, 1024 -> 2 x 2816 1431 and 1434 us; T = 300000,
// 256 -> 2 x 100 500 and 436; T = 65536, 1279 -> 2 x 1365 1003 and 899.
inline Plan token_plan(int64_t N, int64_t M, int64_t kb) {
    Plan p = plan_of(N, M, kb, true, false);
    if (p.pair) p.splits = sum_parts(kb);
    return p;
}

inline bool token_apart(const Plan& p, int64_t kb) { return !p.pair && kb > kSumBlocks * p.splits; }

}  // namespace linear
}  // namespace mhc
