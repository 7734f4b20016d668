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

}  // namespace linear
}  // namespace mhc
