// Matrix product kernels (sm_103a): C[m,n] = sum over k of A[m,k] * B[n,k],
// with scales, bias, activation and residual applied to the FP32 sum before
// its one rounding.  Definitions in mhc_layer.h.  The forward is (m, n, k) =
// (t, o, i), grad_x (t, i, o) and grad_w (o, i, t).
#pragma once

#include "mhc_device.cuh"
#include "mhc_umma.cuh"

namespace mhc {
namespace linear {

constexpr int kE4m3 = 2;   // operand type, beside kBF16 and kF16

enum Act { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3 };

// The normal distribution, from erfc(x) = t (a1 + t (a2 + t (a3 + t (a4 + t
// a5)))) exp(-x^2), t = 1 / (1 + p x), x >= 0 (Abramowitz and Stegun, Handbook
// of Mathematical Functions, 7.1.26: within 1.5e-7), without a branch that
// the lanes of a warp would take apart.
__device__ __forceinline__ float normal_cdf(float z) {
    const float x = fabsf(z) * 0.70710678f;
    const float t = __fdividef(1.0f, __fmaf_rn(0.3275911f, x, 1.0f));
    float q = __fmaf_rn(t, 1.061405429f, -1.453152027f);
    q = __fmaf_rn(t, q, 1.421413741f);
    q = __fmaf_rn(t, q, -0.284496736f);
    q = __fmaf_rn(t, q, 0.254829592f);
    const float tail = 0.5f * q * t * __expf(-x * x);
    return z < 0.0f ? tail : 1.0f - tail;
}

// The forward's exponential is the hardware's (ex2.approx through __expf,
// within a few units of the last FP32 place): the result is rounded to 11
// bits or fewer.
template <int ACT>
__device__ __forceinline__ float activation(float z) {
    if constexpr (ACT == kActRelu) return z <= 0.0f ? 0.0f : z;   // (NaN stays)
    if constexpr (ACT == kActSilu) return __fdividef(z, 1.0f + __expf(-z));
    if constexpr (ACT == kActGelu) return z * normal_cdf(z);
    return z;
}

// The derivatives, with the same exponential: within 2^-20 of the exact ones.
template <int ACT>
__device__ __forceinline__ float slope(float z) {
    if constexpr (ACT == kActRelu) return z > 0.0f ? 1.0f : 0.0f;
    if constexpr (ACT == kActSilu) {
        const float p = __fdividef(1.0f, 1.0f + __expf(-z));
        return p * __fmaf_rn(z, 1.0f - p, 1.0f);
    }
    if constexpr (ACT == kActGelu) return __fmaf_rn(z * 0.39894228f, __expf(-0.5f * z * z), normal_cdf(z));
    return 1.0f;
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
    int64_t a_stride, b_stride;   // of their rows, in elements
    bool a_mn, b_mn;              // rows run along m (n), one for each k; else along k.  b_mn where a_mn.
    bool by_row;                  // a row's sums must not depend on M (its tokens): the forward and grad_x
    int64_t M, N, K;
    Epilogue e;
};

// How the operands P and Q lie in memory: rows along K, or (2-byte types)
// rows along their lanes or columns ("MN-major").
enum Layout { kBothK = 0, kPMnQK = 1, kBothMn = 2 };   // forward, grad_x, grad_w

// How a tile lies: the output's contiguous index n on the lanes of tensor
// memory (operand P = B, 128 lanes a CTA) and its rows m on the columns
// (operand Q = A).  A warp then holds 32 consecutive n of one row, so every
// access of the epilogue is a contiguous 64 bytes whatever the alignment of
// the output, and bias and column scale are one register.
struct TileArgs {
    Epilogue e;
    int64_t N;               // output columns
    uint32_t rows;           // output rows
    uint32_t kb;             // blocks of 128 bytes of K
    uint32_t splits;         // of K; split s takes the blocks [s kb / splits, (s + 1) kb / splits)
    uint32_t width;          // output rows of a tile
    uint32_t stages, stage_bytes;
    uint32_t unit, block_bytes;   // blocks of K of a stage, and bytes of each
    uint32_t idesc;
    uint32_t p_tiles, q_tiles;
    unsigned int* timeouts;
};

constexpr uint32_t kLanesP = 128;                    // lanes of a CTA
constexpr uint32_t kBytesP = kLanesP * 128;          // of one block of K
constexpr uint32_t kPanel = 64 * 128;                // 64 lanes or columns x 64 K, MN-major
constexpr uint32_t kMaxStages = 12;
constexpr uint32_t kKPerBlock = 4;                   // MMAs (32 bytes of K each) of one block

// The residual at rows m0, m0 + step, ... (C of them) of output column n;
// 0 where it is not read.
template <int C>
__device__ __forceinline__ void load_residual(const Epilogue& e, bool n_ok, int64_t n, uint32_t m0, uint32_t step,
                                              uint32_t rows, uint16_t (&r)[C]) {
    if (e.residual == nullptr) return;
    const uint16_t* p = e.residual + int64_t(m0) * e.residual_stride + n;
    const int64_t stride = int64_t(step) * e.residual_stride;
#pragma unroll
    for (int c = 0; c < C; ++c) r[c] = n_ok && m0 + c * step < rows ? ld_stream2(p + c * stride) : uint16_t(0);
}

// From the FP32 sums v of those rows to y (and preact), `at` elements into
// them, rows `stride` bytes apart (Stride: 32 bits where they fit, since a
// 32-bit stride's multiple is added to an address in one instruction).  ALL:
// every row and the column exist; else rows at or past `rows` (the end of the
// output, or of the caller's tile) and, with n_ok false, the whole column are not
// touched.  res: there is a residual.
template <int OUT, int C, bool ALL, typename Stride>
__device__ __forceinline__ void emit(const Epilogue& e, bool res, Stride stride, int64_t at, bool n_ok, uint32_t m0, uint32_t step,
                                     uint32_t rows, float (&v)[C], const uint16_t (&r)[C], float bias, float col_scale) {
    auto there = [&](int c) { return ALL || (n_ok && m0 + c * step < rows); };
    // row c, asked for in order
    auto row = [&](uint16_t*& p, uint32_t c) {
        char* q = reinterpret_cast<char*>(p);
        if (sizeof(Stride) == 4) return reinterpret_cast<uint16_t*>(q + uint64_t(stride) * c);
        p = reinterpret_cast<uint16_t*>(q + stride);
        return reinterpret_cast<uint16_t*>(q);
    };
    if (e.row_scale != nullptr) {
        const float* p = e.row_scale + m0;
#pragma unroll
        for (int c = 0; c < C; ++c, p += step)
            if (there(c)) v[c] = __fmul_rn(__fmul_rn(v[c], __ldg(p)), col_scale);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = __fadd_rn(v[c], bias);
    if (e.preact != nullptr) {
        uint16_t* p = e.preact + at;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            uint16_t* q = row(p, c);
            if (there(c)) *q = Elem<OUT>::cvt(v[c]);
        }
    }
    switch (e.act) {
        case kActRelu:
#pragma unroll
            for (int c = 0; c < C; ++c) v[c] = activation<kActRelu>(v[c]);
            break;
        case kActSilu:
#pragma unroll
            for (int c = 0; c < C; ++c) v[c] = activation<kActSilu>(v[c]);
            break;
        case kActGelu:
#pragma unroll
            for (int c = 0; c < C; ++c) v[c] = activation<kActGelu>(v[c]);
            break;
        default: break;
    }
    if (res) {
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = __fadd_rn(v[c], Elem<OUT>::one(r[c]));
    }
    uint16_t* p = e.y + at;
#pragma unroll
    for (int c = 0; c < C; c += 2) {
        const uint32_t w = Elem<OUT>::pack(v[c], v[c + 1]);
        uint16_t* q = row(p, c);
        if (there(c)) *q = uint16_t(w);
        q = row(p, c + 1);
        if (there(c + 1)) *q = uint16_t(w >> 16);
    }
}

// The same for one chunk by itself, with or without a residual.
template <int OUT, int C>
__device__ __forceinline__ void emit_any(const Epilogue& e, int64_t N, bool n_ok, int64_t n, uint32_t m0, uint32_t step,
                                         uint32_t rows, float (&v)[C], const uint16_t (&r)[C], float bias,
                                         float col_scale) {
    const uint64_t stride = uint64_t(N) * step * 2;
    const int64_t at = int64_t(m0) * N + n;
    const bool res = e.residual != nullptr;
    if (__all_sync(0xFFFFFFFFu, n_ok) && m0 + (C - 1) * step < rows)
        emit<OUT, C, true>(e, res, stride, at, n_ok, m0, step, rows, v, r, bias, col_scale);
    else
        emit<OUT, C, false>(e, res, stride, at, n_ok, m0, step, rows, v, r, bias, col_scale);
}

__device__ __forceinline__ uint32_t split_begin(const TileArgs& a, uint32_t s) {
    return uint32_t(uint64_t(a.kb) * s / a.splits);
}

// One block of K of P (128 lanes from p0) and of Q (`columns` from q0) into a stage.
template <int CG, bool FP8, int LAYOUT>
__device__ __forceinline__ void load_p(uint32_t stage, const CUtensorMap* mp, uint32_t k, int p0, uint32_t bar) {
    const int k0 = int(k * (FP8 ? 128u : 64u));
    if constexpr (LAYOUT == kBothK) {
        umma::tensor_copy_2d<CG>(stage, mp, k0, p0, bar);
    } else {
        umma::tensor_copy_2d<CG>(stage, mp, p0, k0, bar);
        umma::tensor_copy_2d<CG>(stage + kPanel, mp, p0 + 64, k0, bar);
    }
}

template <int CG, bool FP8, int LAYOUT>
__device__ __forceinline__ void load_q(uint32_t stage, const CUtensorMap* mq, uint32_t k, int q0, uint32_t columns,
                                       uint32_t bar) {
    const int k0 = int(k * (FP8 ? 128u : 64u));
    if constexpr (LAYOUT != kBothMn) {
        umma::tensor_copy_2d<CG>(stage + kBytesP, mq, k0, q0, bar);
    } else {
        for (uint32_t j = 0; j < columns; j += 64)
            umma::tensor_copy_2d<CG>(stage + kBytesP + j / 64 * kPanel, mq, q0 + int(j), k0, bar);
    }
}

// Operand descriptors of stage 0; a stage further on adds its bytes / 16.  The
// next 32 bytes of K lie 32 bytes on within the swizzled rows, or, MN-major,
// 16 rows of 128 bytes on (addresses count 16 bytes).
struct Descs {
    uint64_t p, q;
};

template <int LAYOUT>
__device__ __forceinline__ Descs descs(uint32_t stages) {
    return {umma::smem_desc(stages, LAYOUT == kBothK ? 16 : kPanel),
            umma::smem_desc(stages + kBytesP, LAYOUT == kBothMn ? kPanel : 16)};
}

template <int CG, bool FP8, int LAYOUT>
__device__ __forceinline__ void multiply_block(const Descs& d, uint32_t offset, uint32_t idesc, uint32_t tmem, bool first) {
    constexpr uint32_t kP = LAYOUT == kBothK ? 2 : 128, kQ = LAYOUT == kBothMn ? 128 : 2;
    const uint64_t p = d.p + (offset >> 4), q = d.q + (offset >> 4);
#pragma unroll
    for (uint32_t i = 0; i < kKPerBlock; ++i)
        umma::mma<CG, FP8>(tmem, p + i * kP, q + i * kQ, idesc, !(first && i == 0));
}

// The end of a producer, which is at the stage after its last: waits until no
// copy and no completion signal of the last `issued` stages is in flight (for
// their copies alone after a wait that ran out).
__device__ __forceinline__ void drain(bool& ok, uint32_t issued, umma::Ring at, uint32_t count, uint32_t bar_empty,
                                      uint32_t bar_full) {
    for (uint32_t i = 0; i < issued; ++i) {
        if (at.stage == 0) at.stage = count, at.parity ^= 1;
        --at.stage;
        ok = umma::wait((ok ? bar_empty : bar_full) + 8 * at.stage, at.parity) && ok;
    }
}

__device__ __forceinline__ void timed_out(const TileArgs& a) { *a.timeouts = 1u; }

// --------------------------------------------------------------------------
// Few tiles: one tile of 128 lanes x `width` columns a cluster of `splits`
// CTAs, each of which sums its part of K; the parts meet in shared memory and
// are added in increasing order, the columns shared out among the CTAs.
// Bound by the bytes of P where rows are few: one row through 7168 x 7168 20.5
// us (5.0 TB/s), of which about 5 us are the launch, the first copies' latency
// and the join.
//
// Warps 0-15 read tensor memory (four for each quarter of the lanes: 4 warps
// alone took 35 ns a column, 14 us for a 256-row call of 1024 x 1024), warp 16
// copies, warp 17 multiplies.
// --------------------------------------------------------------------------
constexpr uint32_t kEpilogueWarps = 16;
constexpr int kChunk = 8;   // columns that a warp takes out of tensor memory at a time
constexpr uint32_t kSplitThreads = 32 * (kEpilogueWarps + 2);
constexpr uint32_t kSplitCopy = kEpilogueWarps, kSplitMultiply = kSplitCopy + 1;   // warps

template <bool FP8, int OUT, int LAYOUT>
__global__ void __launch_bounds__(kSplitThreads, 1)
split_kernel(const __grid_constant__ CUtensorMap mp, const __grid_constant__ CUtensorMap mq,
             const __grid_constant__ TileArgs a) {
    extern __shared__ char raw[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], done;
    __shared__ uint32_t tmem_base;
    char* stages = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = a.splits > 1 ? umma::cluster_rank() : 0;
    const int64_t n0 = int64_t(blockIdx.x / a.splits) * kLanesP;
    const uint32_t m0 = blockIdx.y * a.width;
    uint32_t columns = 32;
    while (columns < a.width) columns *= 2;
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < a.stages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        mbar_init(&done, 1);
        mbar_init_fence();
    }
    if (warp == kSplitCopy) {
        umma::tmem_alloc<1>(&tmem_base, columns);
        if (lane == 0) {
            umma::prefetch_map(&mp);
            umma::prefetch_map(&mq);
        }
    }
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = tmem_base;
    const uint32_t k0 = split_begin(a, rank), k1 = split_begin(a, rank + 1);
    const uint32_t quarter = warp % 4, group = warp / 4;
    const uint32_t valid = min(a.width, a.rows - m0);
    const int64_t n = n0 + quarter * 32 + lane;
    const bool n_ok = n < a.N;
    // the thread's place in the parts, [column][lane], that take the stages' place
    // once every copy has landed and been read
    float* part = reinterpret_cast<float*>(stages) + quarter * 32 + lane;
    pdl_enter();
    const float bias = a.e.bias != nullptr && n_ok ? __ldg(a.e.bias + n) : 0.0f;
    const float cs = a.e.col_scale != nullptr && n_ok ? __ldg(a.e.col_scale + n) : 1.0f;
    const uint32_t ring = smem_addr(stages), bar_full = smem_addr(full), bar_empty = smem_addr(empty);
    const uint32_t count = a.stages, bytes = a.stage_bytes, unit = a.unit;
    if (warp == kSplitCopy) {
        umma::Ring at;
        bool ok = true;
        uint32_t k = k0, issued = 0;
        for (; k < k1; k += unit, ++issued, at.next(count)) {
            // (the first round finds every stage free: the phase before a new barrier's first one)
            if (!(ok = umma::wait(bar_empty + 8 * at.stage, at.parity ^ 1))) break;
            const uint32_t n = min(unit, k1 - k);
            if (umma::elect()) {
                umma::expect_tx(bar_full + 8 * at.stage, n * a.block_bytes);
                for (uint32_t u = 0; u < n; ++u) {
                    const uint32_t to = ring + at.stage * bytes + u * a.block_bytes;
                    load_p<1, FP8, LAYOUT>(to, &mp, k + u, int(n0), bar_full + 8 * at.stage);
                    load_q<1, FP8, LAYOUT>(to, &mq, k + u, int(m0), a.width, bar_full + 8 * at.stage);
                }
            }
            __syncwarp();
        }
        drain(ok, min(issued, count), at, count, bar_empty, bar_full);
        if (!ok) timed_out(a);
    } else if (warp == kSplitMultiply) {
        const Descs d = descs<LAYOUT>(ring);
        const uint32_t idesc = a.idesc;
        umma::Ring at;
        for (uint32_t k = k0; k < k1; k += unit, at.next(count)) {
            if (!umma::wait(bar_full + 8 * at.stage, at.parity)) {
                timed_out(a);
                break;
            }
            umma::fence_after_sync();
            const uint32_t n = min(unit, k1 - k);
            if (umma::elect()) {
                for (uint32_t u = 0; u < n; ++u)
                    multiply_block<1, FP8, LAYOUT>(d, at.stage * bytes + u * a.block_bytes, idesc, tmem, k + u == k0);
                umma::commit<1>(bar_empty + 8 * at.stage);
                if (k + n == k1) umma::commit<1>(smem_addr(&done));
            }
            __syncwarp();
        }
    } else {
        if (!umma::wait(smem_addr(&done), 0)) timed_out(a);
        umma::fence_after_sync();
        // group g of four warps takes the chunks g, g + 4, ... of the columns
        for (uint32_t c = group * kChunk; c < valid; c += 4 * kChunk) {
            float v[kChunk];
            umma::tmem_ld(tmem + (quarter * 32u << 16) + c, v);
            uint16_t r[kChunk];
            if (a.splits == 1) load_residual<kChunk>(a.e, n_ok, n, m0 + c, 1, m0 + valid, r);
            umma::tmem_wait_ld(v);
            if (a.splits == 1) {
                emit_any<OUT, kChunk>(a.e, a.N, n_ok, n, m0 + c, 1, m0 + valid, v, r, bias, cs);
            } else {
#pragma unroll
                for (int i = 0; i < kChunk; ++i) part[(c + i) * kLanesP] = v[i];
            }
        }
        umma::fence_before_sync();
    }
    __syncwarp();
    if (a.splits > 1) {
        umma::cluster_sync();
        if (warp < kEpilogueWarps) {
            // this CTA's columns are rank, rank + splits, ...; a group takes 8 of
            // them at a time, their loads issued together
            const uint32_t at = smem_addr(part);
            for (uint32_t c = rank + group * kChunk * a.splits; c < valid; c += 4 * kChunk * a.splits) {
                uint16_t res[kChunk];
                load_residual<kChunk>(a.e, n_ok, n, m0 + c, a.splits, m0 + valid, res);
                float v[kChunk];
                for (uint32_t r = 0; r < a.splits; ++r) {
                    const uint32_t peer = umma::map_rank(at, r);
                    float w[kChunk];
#pragma unroll
                    for (uint32_t i = 0; i < kChunk; ++i) {
                        const uint32_t col = c + i * a.splits;
                        w[i] = col < valid ? umma::ld_cluster(peer + col * (kLanesP * 4)) : 0.0f;
                    }
#pragma unroll
                    for (uint32_t i = 0; i < kChunk; ++i) v[i] = r == 0 ? w[i] : __fadd_rn(v[i], w[i]);
                }
                emit_any<OUT, kChunk>(a.e, a.N, n_ok, n, m0 + c, a.splits, m0 + valid, v, res, bias, cs);
            }
        }
        umma::cluster_sync();   // no CTA leaves while another reads its part
    } else {
        __syncthreads();
    }
    umma::fence_after_sync();
    if (warp == kSplitCopy) umma::tmem_free<1>(tmem, columns);
}

// --------------------------------------------------------------------------
// Many tiles: a pair of CTAs on two SMs computes tiles of 256 lanes x `width`
// columns (each holds half the lanes of P and half the columns of Q in its
// shared memory, and half the lanes of the sums), one after the other, the
// copies running ahead across tiles.  Two accumulators of `width` columns
// alternate, so the epilogue of one tile runs under the multiplication of the
// next.  The parts of K that split_kernel gives to different CTAs are summed
// apart here too and added in the same order, so that both kernels give the
// same bits (PARTS): the second part's accumulator takes the others' sums in,
// the first one holds every other part.  (Sums in registers instead, 64 or
// 128 columns a thread, spilled: T = 4096, 7168 x 7168 269 to 330 us.)  Bound by
// the tensor cores and their power: T = 4096, 7168 x 7168 225 us (1870 TFLOP/s)
// in short runs, with bias, gelu and residual 278 us in long ones.
//
// Warps 0-15 read tensor memory (four warps for each quarter of the lanes, a
// quarter of the columns each).  Warp 16 copies P, warp 18 copies Q (a block of K
// has 512 cycles, of which a copy and its wait take well over 100), warp 17 (of
// the first CTA) multiplies.
// --------------------------------------------------------------------------
constexpr uint32_t kPairThreads = 32 * (kEpilogueWarps + 3);
constexpr uint32_t kCopyP = kEpilogueWarps, kMultiply = kCopyP + 1, kCopyQ = kCopyP + 2;   // warps
constexpr uint32_t kTmemColumns = 512;

// Tile i of the order: bands of kBand p tiles, in each band q tile by q tile,
// so that the tiles in flight share their operands in L2.
constexpr uint32_t kBand = 8;


__device__ __forceinline__ void tile_at(const TileArgs& a, uint32_t i, uint32_t& p, uint32_t& q) {
    const uint32_t band = i / (kBand * a.q_tiles);
    const uint32_t first = band * kBand;
    const uint32_t height = min(kBand, a.p_tiles - first);
    const uint32_t j = i - first * a.q_tiles;
    q = j / height;
    p = first + (j - q * height);
}

// The accumulator of each part of each tile in turn, and the parity of its
// round (one bit each): as many rounds as it was taken before.
struct Sums {
    uint32_t rounds = 3, last = 1;
    // (PARTS: the second part's is the second one, every other part's the first)
    template <bool PARTS>
    __device__ __forceinline__ uint32_t take(uint32_t part) {
        last = PARTS ? uint32_t(part == 1) : last ^ 1;
        rounds ^= 1u << last;
        return last;
    }
    __device__ __forceinline__ uint32_t parity(uint32_t b) const { return rounds >> b & 1; }
};

// A warp's `mine` columns of a finished tile, from tensor memory at `from`.
// The next chunk's sums and residual arrive while a chunk is worked on;
// give_back after the last read of tensor memory.  Short K is bound by the
// instructions here: the checks once a tile and 32-bit strides took T = 10388, 128 x
// 11048 from 86 to 72 us (3.2 TB/s of output).
template <int OUT, bool ALL, bool RES, typename GiveBack>
__device__ __forceinline__ void emit_tile(const TileArgs& a, uint32_t from, uint32_t mine, uint32_t m0, int64_t col, bool n_ok,
                                          float bias, float cs, GiveBack give_back) {
    uint16_t r[kChunk];
    if constexpr (RES) load_residual<kChunk>(a.e, n_ok, col, m0, 1, a.rows, r);
    float next[kChunk];
    umma::tmem_ld(from, next);
    int64_t at = int64_t(m0) * a.N + col;
#pragma unroll 1
    for (uint32_t c = 0; c < mine; c += kChunk, at += kChunk * a.N) {
        umma::tmem_wait_ld(next);
        float v[kChunk];
        uint16_t now[kChunk];
#pragma unroll
        for (int k = 0; k < kChunk; ++k) v[k] = next[k], now[k] = RES ? r[k] : uint16_t(0);
        if (c + kChunk < mine) {
            umma::tmem_ld(from + c + kChunk, next);
            if constexpr (RES) load_residual<kChunk>(a.e, n_ok, col, m0 + c + kChunk, 1, a.rows, r);
        } else {
            give_back();
        }
        emit<OUT, kChunk, ALL>(a.e, RES, uint32_t(a.N) * 2u, at, n_ok, m0 + c, 1, a.rows, v, now, bias, cs);
    }
}

template <bool FP8, int OUT, int LAYOUT, bool PARTS>
__global__ void __launch_bounds__(kPairThreads, 1)
pair_kernel(const __grid_constant__ CUtensorMap mp, const __grid_constant__ CUtensorMap mq,
            const __grid_constant__ TileArgs a) {
    extern __shared__ char raw[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], sum_full[2], sum_empty[2];
    __shared__ uint32_t tmem_base;
    char* stages = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = umma::cluster_rank();
    const uint32_t half = a.width / 2;
    const uint32_t tiles = a.p_tiles * a.q_tiles, step = gridDim.x / 2;
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < a.stages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(sum_full + b, 1);
            mbar_init(sum_empty + b, 2 * kEpilogueWarps);
        }
        mbar_init_fence();
    }
    if (warp == kCopyP) {
        umma::tmem_alloc<2>(&tmem_base, kTmemColumns);
        if (lane == 0) {
            umma::prefetch_map(&mp);
            umma::prefetch_map(&mq);
        }
    }
    umma::fence_before_sync();
    __syncthreads();
    umma::cluster_sync();   // the other CTA's barriers are ready too
    umma::fence_after_sync();
    const uint32_t tmem = tmem_base;
    pdl_enter();
    const uint32_t ring = smem_addr(stages), bar_full = smem_addr(full), bar_empty = smem_addr(empty);
    const uint32_t bar_sum = smem_addr(sum_full), bar_free = smem_addr(sum_empty);
    const uint32_t count = a.stages, bytes = a.stage_bytes, unit = a.unit;
    if (warp == kCopyP || warp == kCopyQ) {
        // both CTAs' copies count on the first one's barrier; its phase cannot end
        // before that CTA's arrival, whichever copy lands first
        const uint32_t bar_pair = umma::map_rank(bar_full, 0);
        umma::Ring at;
        bool ok = true;
        uint32_t issued = 0;
        for (uint32_t i = blockIdx.x / 2; i < tiles && ok; i += step) {
            uint32_t pt, qt;
            tile_at(a, i, pt, qt);
            const int p0 = int(pt * 2 * kLanesP + rank * kLanesP), q0 = int(qt * a.width + rank * half);
            uint32_t k = 0;
            for (uint32_t part = 0; part < a.splits && ok; ++part) {
                for (const uint32_t k1 = split_begin(a, part + 1); k < k1; ++issued, at.next(count)) {
                    if (!(ok = umma::wait(bar_empty + 8 * at.stage, at.parity ^ 1))) break;
                    const uint32_t n = min(unit, k1 - k);
                    if (umma::elect()) {
                        if (warp == kCopyP && rank == 0) umma::expect_tx(bar_full + 8 * at.stage, 2 * n * a.block_bytes);
                        for (uint32_t u = 0; u < n; ++u) {
                            const uint32_t to = ring + at.stage * bytes + u * a.block_bytes;
                            if (warp == kCopyP) load_p<2, FP8, LAYOUT>(to, &mp, k + u, p0, bar_pair + 8 * at.stage);
                            else load_q<2, FP8, LAYOUT>(to, &mq, k + u, q0, half, bar_pair + 8 * at.stage);
                        }
                    }
                    __syncwarp();
                    k += n;
                }
            }
        }
        drain(ok, min(issued, count), at, count, bar_empty, rank == 0 ? bar_full : bar_empty);
        if (!ok) timed_out(a);
    } else if (warp == kMultiply) {
        if (rank == 0) {
            const Descs d = descs<LAYOUT>(ring);
            const uint32_t idesc = a.idesc;
            umma::Ring at;
            Sums sums;
            bool ok = true;
            for (uint32_t i = blockIdx.x / 2; i < tiles && ok; i += step) {
                uint32_t k = 0;
                for (uint32_t part = 0; part < a.splits && ok; ++part) {
                    const uint32_t b = sums.take<PARTS>(part);
                    if (!(ok = umma::wait(bar_free + 8 * b, sums.parity(b) ^ 1))) break;
                    umma::fence_after_sync();
                    const uint32_t to = tmem + b * 256, k0 = k, k1 = split_begin(a, part + 1);
                    for (; k < k1; at.next(count)) {
                        if (!(ok = umma::wait(bar_full + 8 * at.stage, at.parity))) break;
                        umma::fence_after_sync();
                        const uint32_t n = min(unit, k1 - k);
                        if (umma::elect()) {
                            for (uint32_t u = 0; u < n; ++u)
                                multiply_block<2, FP8, LAYOUT>(d, at.stage * bytes + u * a.block_bytes, idesc, to, k + u == k0);
                            umma::commit<2>(bar_empty + 8 * at.stage);
                            if (k + n == k1) umma::commit<2>(bar_sum + 8 * b);
                        }
                        __syncwarp();
                        k += n;
                    }
                }
            }
            if (!ok) timed_out(a);
        }
    } else {
        const uint32_t quarter = warp % 4, mine = a.width / 4, c0 = warp / 4 * mine;   // its columns: c0 .. c0 + mine
        const uint32_t tw = tmem + (quarter * 32u << 16) + c0;
        const uint32_t signal = umma::map_rank(bar_free, 0);
        Sums sums;
        bool ok = true;
        for (uint32_t i = blockIdx.x / 2; i < tiles && ok; i += step) {
            uint32_t pt, qt;
            tile_at(a, i, pt, qt);
            const int64_t col = int64_t(pt) * 2 * kLanesP + rank * kLanesP + quarter * 32 + lane;
            const uint32_t m0 = qt * a.width + c0;
            const bool n_ok = col < a.N;
            const float bias = a.e.bias != nullptr && col < a.N ? __ldg(a.e.bias + col) : 0.0f;
            const float cs = a.e.col_scale != nullptr && col < a.N ? __ldg(a.e.col_scale + col) : 1.0f;
            // the warp's residual (64 bytes of each row) to L2, under the multiplication:
            // a chunk at a time from memory took 2400 cycles each
            if (a.e.residual != nullptr) {
                const int64_t col0 = col - lane;
                for (uint32_t c = lane; c < mine; c += 32)
                    if (m0 + c < a.rows && col0 < a.N) umma::prefetch_l2(a.e.residual + int64_t(m0 + c) * a.e.residual_stride + col0);
            }
            uint32_t b = 0;
            for (uint32_t part = 0; part < a.splits; ++part) {
                b = sums.take<PARTS>(part);
                if (!(ok = umma::wait(bar_sum + 8 * b, sums.parity(b)))) break;
                umma::fence_after_sync();
                if (!PARTS || part == 0) continue;
                // the second accumulator becomes the sum of the parts so far
#pragma unroll 2
                for (uint32_t c = 0; c < mine; c += kChunk) {
                    float v[kChunk], w[kChunk];
                    umma::tmem_ld(tw + c, v);
                    umma::tmem_ld(tw + 256 + c, w);
                    umma::tmem_wait_ld(v);
                    umma::tmem_wait_ld(w);
                    // (the second part arrives where the sum goes)
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) v[i] = __fadd_rn(v[i], w[i]);
                    umma::tmem_st(tw + 256 + c, v);
                }
                umma::tmem_wait_st();
                umma::fence_before_sync();
                __syncwarp();
                if (lane == 0) umma::arrive_cluster(signal);
                b = 1;
            }
            if (!ok) break;
            auto give_back = [&] {
                umma::fence_before_sync();
                __syncwarp();
                if (lane == 0) umma::arrive_cluster(signal + 8 * b);
            };
            // (the same for the whole warp)
            const bool all = __all_sync(0xFFFFFFFFu, n_ok) && m0 + mine <= a.rows;
            if (a.e.residual != nullptr) {
                if (all) emit_tile<OUT, true, true>(a, tw + b * 256, mine, m0, col, n_ok, bias, cs, give_back);
                else emit_tile<OUT, false, true>(a, tw + b * 256, mine, m0, col, n_ok, bias, cs, give_back);
            } else {
                if (all) emit_tile<OUT, true, false>(a, tw + b * 256, mine, m0, col, n_ok, bias, cs, give_back);
                else emit_tile<OUT, false, false>(a, tw + b * 256, mine, m0, col, n_ok, bias, cs, give_back);
            }
        }
        if (!ok) timed_out(a);
        umma::fence_before_sync();
    }
    __syncwarp();
    umma::cluster_sync();   // neither CTA leaves while the other may still signal it
    umma::fence_after_sync();
    if (warp == kCopyP) umma::tmem_free<2>(tmem, kTmemColumns);
}

// Rows of values copied to a row pitch that starts every row on 16 bytes, for
// operands that the tensor copies cannot read in place: up to two of them in
// one launch.  A thread writes one 16-byte vector from the two aligned ones
// that hold its bytes (one by one where those reach outside the source).
struct Repack {
    const char* src;
    char* dst;
    uint64_t vectors;            // of all rows
    uint32_t per_row;            // vectors of a row at dst
    FastDivU32 by_row;
    uint64_t length, stride;     // bytes of a row and between rows
    uint64_t bytes;              // of src, from the first row's start to the last one's end
};

constexpr uint32_t kRepackThreads = 256;

static __global__ void __launch_bounds__(kRepackThreads) repack_kernel(const Repack first, const Repack second, uint32_t blocks) {
    pdl_enter();
    const bool one = blockIdx.x < blocks;
    const Repack& r = one ? first : second;
    const uint64_t i = uint64_t(one ? blockIdx.x : blockIdx.x - blocks) * kRepackThreads + threadIdx.x;
    if (i >= r.vectors) return;
    const uint64_t row = r.vectors <= 0xFFFFFFFFull ? fastdiv_u32(uint32_t(i), r.by_row) : i / r.per_row;
    const uint64_t c = (i - row * r.per_row) * 16;         // byte within the row
    const char* p = r.src + row * r.stride + c;
    const uint32_t shift = uint32_t(reinterpret_cast<uintptr_t>(p) & 15u);
    const char* base = p - shift;
    uint32_t w[8];
    if (base >= r.src && base + 32 <= r.src + r.bytes) {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(base)), b = __ldg(reinterpret_cast<const uint4*>(base) + 1);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
        // whole words first, then the rest of the shift
#pragma unroll
        for (int s = 2; s > 0; s >>= 1)
            if ((shift / 4) & s) {
#pragma unroll
                for (int k = 0; k + s < 8; ++k) w[k] = w[k + s];
            }
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 8 * (shift & 3u));
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            w[k] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + 4 * k + j < r.length) w[k] |= uint32_t(static_cast<uint8_t>(__ldg(p + 4 * k + j))) << (8 * j);
        }
    }
    // (bytes past the row's end are read by nobody: the tensor map ends with the row)
    *reinterpret_cast<uint4*>(r.dst + i * 16) = make_uint4(w[0], w[1], w[2], w[3]);
}

// u = g * act'(preact) over [T,O], rounded to u (row pitch `pitch`; null: not stored), and the
// column sums of the unrounded u over each of gridDim.y runs of `rows` rows
// in partial [gridDim.y, O] (null: not wanted).  u is rounded to the storage type since both
// products read it as an operand of the tensor cores, which take 16 bits: BF16 grad_x and
// grad_w are then 2.35e-3 off in norm (1.66e-3 is their own last rounding; T = 4096, 4096 x
// 7168, silu); a second operand for the rest of u would double the products' work.
// Block (32, 8): 32 W columns,
// 8 rows at a time.  HBM-bound: T = 4096, O = 7168 29 us (176 MB, 90% of the copy
// bandwidth; 50 us with the exact division and exponential).
constexpr int kSlopeRows = 8;

template <int W>
struct Row;

template <>
struct Row<8> {
    Words<4> w;
    __device__ __forceinline__ void load(const uint16_t* p) { w = ld_stream<4>(p); }
    template <int DT>
    __device__ __forceinline__ float value(int i) const {
        return i % 2 ? Elem<DT>::hi(w.w[i / 2]) : Elem<DT>::lo(w.w[i / 2]);
    }
};

template <>
struct Row<1> {
    uint16_t w;
    __device__ __forceinline__ void load(const uint16_t* p) { w = ld_stream2(p); }
    template <int DT>
    __device__ __forceinline__ float value(int) const { return Elem<DT>::one(w); }
};

template <int DT, int W>
__device__ __forceinline__ void store_row(uint16_t* p, const float (&v)[W]) {
    if constexpr (W == 8) {
        Words<4> o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o.w[i] = Elem<DT>::pack(v[2 * i], v[2 * i + 1]);
        *reinterpret_cast<Words<4>*>(p) = o;
    } else {
        *p = Elem<DT>::cvt(v[0]);
    }
}

template <int DT, int W, int ACT>
__global__ void __launch_bounds__(32 * kSlopeRows, 4)
slope_kernel(const uint16_t* __restrict__ g, const uint16_t* __restrict__ preact, uint16_t* __restrict__ u,
             float* __restrict__ partial, int64_t T, int64_t O, int64_t pitch, int64_t rows) {
    pdl_enter();
    __shared__ float part[kSlopeRows][32 * W];
    const int64_t c = (int64_t(blockIdx.x) * 32 + threadIdx.x) * W;
    const int64_t t0 = int64_t(blockIdx.y) * rows, t1 = min(t0 + rows, T);
    float acc[W];
#pragma unroll
    for (int i = 0; i < W; ++i) acc[i] = 0.0f;
    // two rows' loads are under way together, in four blocks an SM: T = 16000, O = 2048
    // 35 us, with four rows and three blocks 42
    constexpr int kAhead = 2;
    for (int64_t t = t0 + threadIdx.y; t < t1 && c < O; t += kAhead * kSlopeRows) {
        Row<W> gr[kAhead], zr[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (t + k * kSlopeRows < t1) {
                const int64_t at = (t + k * kSlopeRows) * O + c;
                gr[k].load(g + at);
                if (ACT != kActNone) zr[k].load(preact + at);
            }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (t + k * kSlopeRows < t1) {
                float v[W];
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    v[i] = gr[k].template value<DT>(i);
                    if (ACT != kActNone) v[i] *= slope<ACT>(zr[k].template value<DT>(i));
                    acc[i] = __fadd_rn(acc[i], v[i]);
                }
                if (u != nullptr) store_row<DT>(u + (t + k * kSlopeRows) * pitch + c, v);
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
