// RMS norm kernels (sm_103a): forward with the residual's addition and an
// optional 8-bit output, and backward.  Definitions in mhc_layer.h.
//
// HBM-bound: about 5 operations per value that is read or written once.  A
// row is held in registers between the sum of squares and the output, so each
// value crosses HBM once.  Measured at H = 7168 with the residual, of the
// copy bandwidth: T = 65536 with 8-bit output 513 us (96%), T = 4096 38.9 us
// (90%; its start and its last rows are the rest), backward T = 4096 47.0 us
// (75%: one block an SM, whose rows follow one another through two passes and
// a barrier, and the column sums' launch after it).
//
// Order of a row's sum (it depends on H only): the row is cut into chunks of
// 8 values; thread j of the row's nt threads owns chunks j, j + nt, ... (at
// most K of them), sums each as the pairwise tree ((0+1)+(2+3))+((4+5)+(6+7))
// and adds the chunks in increasing order; a warp folds by exchanging with
// lanes at distance 16, 8, 4, 2, 1; the warps' results are added pairwise
// (0+1)+(2+3), ....  nt and K follow from H (shape_of).
//
// Values are worked on in packed pairs (mhc_f32x2.cuh): half the instructions
// of a row's chain.  No packed product is an operand of a packed sum that is
// not written as one fused multiply-add here, so that every kernel rounds
// alike.
//
// Three ways to move a row, with the same sums:
//  * ring: rows of 16-byte aligned values (H % 8 == 0) longer than a warp
//    holds, more of them than there are blocks: bulk copies bring a block's
//    next rows to shared memory while it works on one, so that the loads of
//    a row do not wait for its sum; the norm's weight stays in registers;
//  * VEC: 16-byte loads and stores of the thread's own chunks, for the other
//    aligned rows;
//  * otherwise (odd H, strides or pointers off 16 bytes) the same chunks, each
//    from the two aligned vectors that hold it, and to aligned vectors put
//    together from two neighbouring lanes' chunks; the row's ends go value by value.  (Moving single values, a thread taking j, j +
//    nt, ..., and exchanging the sums' terms through shared memory: T = 20000,
//    H = 1279 109 us, backward 113.)
#pragma once

#include "mhc_bulk.cuh"
#include "mhc_device.cuh"
#include "mhc_f32x2.cuh"

namespace mhc {
namespace norm {

constexpr int kMaxH = 32768;
constexpr int kMaxThreads = 512;   // of a row
constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 0x1p-60f;

enum Out { kOutSame = 0, kOutFp8Row = 1, kOutFp8Group = 2 };
constexpr int kGroup = 128;

struct FwdArgs {
    const uint16_t* x;
    const uint16_t* residual;   // null without one
    const float* weight;
    void* y;
    float* scale;
    uint16_t* total;
    float* rstd;
    unsigned int* timeouts;     // ring kernels only
    int64_t T;
    int64_t x_stride, residual_stride;
    uint32_t H;
    float eps;
};

struct BwdArgs {
    const uint16_t* g;
    const uint16_t* s;
    const float* weight;
    const float* rstd;
    const uint16_t* grad_total;   // null without one
    uint16_t* grad_x;
    float* partial;               // [gridDim.x, pitch]
    uint32_t pitch;
    unsigned int* timeouts;       // ring kernels only
    int64_t T;
    int64_t g_stride, s_stride;
    uint32_t H;
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Two E4M3 values, rounded to nearest even; past 448 they stay at 448.
__device__ __forceinline__ uint16_t e4m3_pair(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Folds one value per thread over the row's threads (a warp, or the block):
// every thread gets the result.  `shared` is free again after the caller's
// next barrier; the warps' results meet in a pairwise tree, read four at a
// time (one after the other they took 35 cycles each).
constexpr int kMaxWarps = kMaxThreads / 32;

struct Fold {
    float4 v[kMaxWarps / 4];
};

// The places of warps that the row does not have hold zeros, which change no
// sum and no maximum of magnitudes.  Before the first fold, with a barrier
// between or the fold's own.
__device__ __forceinline__ void clear_fold(Fold* f, int count) {
    if (blockDim.x > 32)
        for (int i = threadIdx.x; i < count * kMaxWarps; i += blockDim.x)
            if (i % kMaxWarps >= int(blockDim.x >> 5)) reinterpret_cast<float*>(f)[i] = 0.0f;
}

template <class Op>
__device__ __forceinline__ float fold(float v, Fold& shared, Op op) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    if (blockDim.x == 32) return v;
    if ((threadIdx.x & 31u) == 0) reinterpret_cast<float*>(&shared)[threadIdx.x >> 5] = v;
    __syncthreads();
    float t[kMaxWarps / 4];
#pragma unroll
    for (int i = 0; i < kMaxWarps / 4; ++i) {
        const float4 x = shared.v[i];
        t[i] = op(op(x.x, x.y), op(x.z, x.w));
    }
    return op(op(t[0], t[1]), op(t[2], t[3]));
}

struct Add {
    __device__ float operator()(float a, float b) const { return __fadd_rn(a, b); }
};
struct Max {
    __device__ float operator()(float a, float b) const { return max_nan(a, b); }
};

// The bytes `shift` .. shift + 4 N - 1 (shift at most 4 N) of the 8 N bytes in
// w, to its first N words: by words with selects (a branch on the words, the
// same for the whole row, kept the loads of a row's chunks from going out
// together: T = 20000, H = 1279 61 -> 82 us), then by the rest.
template <int N>
__device__ __forceinline__ void shift_bytes(uint32_t (&w)[2 * N], uint32_t shift) {
    const uint32_t words = shift / 4;
#pragma unroll
    for (int s = N; s > 0; s >>= 1)
        if (words & s) {
#pragma unroll
            for (int k = 0; k + s < 2 * N; ++k) w[k] = w[k + s];
        }
#pragma unroll
    for (int k = 0; k < N; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 8 * (shift & 3u));
}

// An input of 2-byte rows, and where its first row starts and its last ends.
struct Input {
    const uint16_t* p;
    int64_t stride;
    const char *lo, *hi;
    __device__ __forceinline__ Input(const uint16_t* ptr, int64_t row_stride, int64_t T, uint32_t H)
        : p(ptr),
          stride(row_stride),
          lo(reinterpret_cast<const char*>(ptr)),
          hi(reinterpret_cast<const char*>(ptr + (T - 1) * row_stride + H)) {}
};

// One row in the registers of the row's threads; values past H read as +0.
template <int K, bool VEC>
__device__ __forceinline__ void load_words(const Input& in, int64_t t, uint32_t H, Words<4> (&w)[K]) {
    const uint16_t* row = in.p + t * in.stride;
    const uint32_t nt = blockDim.x, j = threadIdx.x;
    if constexpr (VEC) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint32_t c = 8 * (j + k * nt);
            if (c < H) {
                w[k] = ld_stream<4>(row + c);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) w[k].w[i] = 0;
            }
        }
    } else {
        const uint32_t shift = uint32_t(reinterpret_cast<uintptr_t>(row) & 15u);
        const char* base = reinterpret_cast<const char*>(row) - shift;
        uint32_t v[K][8];
        const bool inside = base >= in.lo && base + 2 * uint64_t(H) + 32 <= in.hi;   // with every vector of the row
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint32_t c = 8 * (j + k * nt);
            const char* q = base + 2 * c;
            if (c < H && (inside || (q >= in.lo && q + 32 <= in.hi))) {
                const uint4 x = __ldg(reinterpret_cast<const uint4*>(q)), y = __ldg(reinterpret_cast<const uint4*>(q) + 1);
                v[k][0] = x.x, v[k][1] = x.y, v[k][2] = x.z, v[k][3] = x.w;
                v[k][4] = y.x, v[k][5] = y.y, v[k][6] = y.z, v[k][7] = y.w;
            } else {   // past the row, or a vector that is not all inside the input: at the shift's place
#pragma unroll
                for (int i = 0; i < 8; ++i) v[k][i] = 0;
                if (c < H) {
                    uint32_t one[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (c + i < H) one[i / 2] |= uint32_t(__ldg(row + c + i)) << (16 * (i & 1));
                    // (shift_bytes below moves them back down)
                    uint32_t up[8] = {0, 0, 0, 0, one[0], one[1], one[2], one[3]};
                    shift_bytes<4>(up, 16 - shift);
                    uint32_t high[8] = {one[0], one[1], one[2], one[3], 0, 0, 0, 0};
                    shift_bytes<4>(high, 16 - shift);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[k][i] = up[i], v[k][4 + i] = high[i];
                }
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            shift_bytes<4>(v[k], shift);
            const uint32_t c = 8 * (j + k * nt);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[k].w[i] = v[k][i];
            if (c < H && c + 8 > H) {   // the row's last chunk
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + 2 * i + 1 >= H) w[k].w[i] &= c + 2 * i >= H ? 0u : 0xFFFFu;
            }
        }
    }
}

__device__ __forceinline__ F2 pfma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

template <int DT>
__device__ __forceinline__ F2 pair_of(uint32_t w) { return f2(Elem<DT>::lo(w), Elem<DT>::hi(w)); }

// A chunk's sum of four packed products, in the chunk's tree.
__device__ __forceinline__ float chunk_sum(const F2 (&q)[4]) {
    return __fadd_rn(__fadd_rn(padd_halves(q[0]), padd_halves(q[1])), __fadd_rn(padd_halves(q[2]), padd_halves(q[3])));
}

// The values lo .. hi - 1 of the 8 that v would put at the aligned address `at`.
template <int SIZE>
__device__ __forceinline__ void put_some(char* at, const uint32_t* v, uint32_t lo, uint32_t hi) {
    for (uint32_t i = lo; i < hi; ++i) {
        if constexpr (SIZE == 2) {
            const uint32_t x = i & 4 ? (i & 2 ? v[3] : v[2]) : (i & 2 ? v[1] : v[0]);
            st_stream2(at + 2 * i, uint16_t(i & 1 ? x >> 16 : x));
        } else {
            at[i] = char((i & 4 ? v[1] : v[0]) >> (8 * (i & 3)));
        }
    }
}

// The words of a row's last lanes' chunks, for the first lanes of the warps
// after them: written before a barrier, read after it.
constexpr int kEdges = kMaxThreads / 32 * 8;   // warps x chunks, at most

template <int N, int K>
__device__ __forceinline__ void publish_edges(uint4* edge, const uint32_t (&w)[K][N]) {
    if (blockDim.x == 32 || (threadIdx.x & 31u) != 31) return;
#pragma unroll
    for (int k = 0; k < K; ++k)
        edge[k * (blockDim.x >> 5) + (threadIdx.x >> 5)] = make_uint4(w[k][0], w[k][1], N > 2 ? w[k][N - 2] : 0, N > 2 ? w[k][N - 1] : 0);
}

// A row whose chunks (8 values of SIZE bytes in N = 2 SIZE words) need not be
// aligned.  The aligned vector that a chunk's first values lie in begins with
// the last `off` values of the chunk before it: the previous lane's, for a
// warp's first lane the previous warp's (edge) or its own last lane's.  A
// vector that the row's start or end cuts is written value by value.
template <int SIZE, int K>
__device__ __forceinline__ void store_unaligned(char* row, uint32_t H, const uint32_t (&w)[K][2 * SIZE], const uint4* edge) {
    constexpr int N = 2 * SIZE;
    const uint32_t lane = threadIdx.x & 31u, warps = blockDim.x >> 5;
    const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(row) & (8 * SIZE - 1)) / SIZE;   // values
    char* base = row - off * SIZE;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const uint32_t c = 8 * (threadIdx.x + k * blockDim.x);
        uint32_t v[2 * N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = __shfl_up_sync(0xFFFFFFFFu, w[k][i], 1);
            v[N + i] = w[k][i];
            if (warps == 1 && k > 0) {
                const uint32_t last = __shfl_sync(0xFFFFFFFFu, w[k > 0 ? k - 1 : 0][i], 31);
                if (lane == 0) v[i] = last;
            }
        }
        if (warps > 1 && lane == 0 && c > 0) {
            const uint4 x = edge[k * warps + (threadIdx.x >> 5) - 1];
            v[0] = x.x, v[1] = x.y;
            if constexpr (N > 2) v[2] = x.z, v[3] = x.w;
        }
        shift_bytes<N>(v, 8 * SIZE - off * SIZE);
        char* at = base + uint64_t(c) * SIZE;
        if (c < H + off) {
            const uint32_t lo = c == 0 ? off : 0, hi = min(8u, H + off - c);
            if (hi - lo == 8) {
                if constexpr (SIZE == 2) __stcs(reinterpret_cast<uint4*>(at), make_uint4(v[0], v[1], v[2], v[3]));
                else __stcs(reinterpret_cast<uint2*>(at), make_uint2(v[0], v[1]));
            } else {
                put_some<SIZE>(at, v, lo, hi);
            }
        }
    }
    // past the last thread's last chunk
    const uint32_t c = 8 * blockDim.x * K;
    if (threadIdx.x + 1 == blockDim.x && c < H + off) {
        uint32_t v[2 * N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = w[K - 1][i], v[N + i] = 0;
        shift_bytes<N>(v, 8 * SIZE - off * SIZE);
        put_some<SIZE>(base + uint64_t(c) * SIZE, v, 0, H + off - c);
    }
}

template <int DT, int K>
__device__ __forceinline__ void pack_row(const F2 (&v)[4 * K], uint32_t (&w)[K][4]) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[k][i] = Elem<DT>::pack(f2_lo(v[4 * k + i]), f2_hi(v[4 * k + i]));
}

template <int K>
__device__ __forceinline__ void store_aligned(uint16_t* __restrict__ row, uint32_t H, const uint32_t (&w)[K][4]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const uint32_t c = 8 * (threadIdx.x + k * blockDim.x);
        if (c < H) __stcs(reinterpret_cast<uint4*>(row + c), make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]));
    }
}

// (without VEC with a barrier inside, for rows of more than one warp)
template <int DT, int K, bool VEC>
__device__ __forceinline__ void store_row(uint16_t* __restrict__ row, uint32_t H, const F2 (&v)[4 * K], uint4* edge) {
    uint32_t w[K][4];
    pack_row<DT, K>(v, w);
    if constexpr (VEC) {
        store_aligned<K>(row, H, w);
    } else {
        publish_edges<4, K>(edge, w);
        if (blockDim.x > 32) __syncthreads();
        store_unaligned<2, K>(reinterpret_cast<char*>(row), H, w, edge);
    }
}

// The norm's weight at the thread's values (it stays in L1: 4 H bytes).
template <int K, bool VEC>
__device__ __forceinline__ void load_weight(const float* __restrict__ w, uint32_t H, F2 (&v)[4 * K]) {
    const uint32_t nt = blockDim.x, j = threadIdx.x;
    const bool vectors = VEC || (reinterpret_cast<uintptr_t>(w) & 15u) == 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const uint32_t c = 8 * (j + k * nt);
        if (vectors && c + (VEC ? 0 : 7) < H) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(w + c)), b = __ldg(reinterpret_cast<const float4*>(w + c) + 1);
            v[4 * k] = f2(a.x, a.y), v[4 * k + 1] = f2(a.z, a.w), v[4 * k + 2] = f2(b.x, b.y), v[4 * k + 3] = f2(b.z, b.w);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[4 * k + i] = f2(!VEC && c + 2 * i < H ? __ldg(w + c + 2 * i) : 0.0f,
                                  !VEC && c + 2 * i + 1 < H ? __ldg(w + c + 2 * i + 1) : 0.0f);
        }
    }
}

// The thread's part of the row's sum of squares.
template <int K>
__device__ __forceinline__ float squares(const F2 (&s)[4 * K]) {
    float acc = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        F2 q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = pmul(s[4 * k + i], s[4 * k + i]);
        acc = __fadd_rn(acc, chunk_sum(q));
    }
    return acc;
}

__device__ __forceinline__ float rstd_of(float sum, uint32_t H, float eps) {
    return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sum, float(H)), eps)));
}

template <int K>
__device__ __forceinline__ void normalise(F2 (&s)[4 * K], float rstd, const F2 (&w)[4 * K]) {
    const F2 r = f2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < 4 * K; ++i) s[i] = pmul(pmul(s[i], r), w[i]);
}

// The row's output from v: 16-bit values, or E4M3 values and their scales.
template <int DT, int K, bool VEC, int OUT>
__device__ __forceinline__ void store_y(const FwdArgs& a, int64_t t, const F2 (&v)[4 * K], Fold& shared, uint4* edge) {
    const uint32_t H = a.H, nt = blockDim.x, j = threadIdx.x;
    if constexpr (OUT == kOutSame) {
        store_row<DT, K, VEC>(static_cast<uint16_t*>(a.y) + t * int64_t(H), H, v, edge);
    } else {
        uint8_t* y = static_cast<uint8_t*>(a.y) + t * int64_t(H);
        float s[8 * K];
#pragma unroll
        for (int i = 0; i < 4 * K; ++i) s[2 * i] = f2_lo(v[i]), s[2 * i + 1] = f2_hi(v[i]);
        float inv[K];   // of the thread's chunks
        if constexpr (OUT == kOutFp8Row) {
            float m = kAmaxFloor;
#pragma unroll
            for (int i = 0; i < 8 * K; ++i) m = max_nan(m, fabsf(s[i]));
            m = fold(m, shared, Max());
            if (j == 0) a.scale[t] = __fdiv_rn(m, kE4m3Max);
            const float r = __fdiv_rn(kE4m3Max, m);
#pragma unroll
            for (int k = 0; k < K; ++k) inv[k] = r;
        } else {
            // 16 chunks to a group: half a warp's chunks of the same k
            const uint32_t groups = (H + kGroup - 1) / kGroup;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float m = kAmaxFloor;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(s[8 * k + i]));
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
                inv[k] = __fdiv_rn(kE4m3Max, m);
                const uint32_t c = j + k * nt;
                if ((j & 15u) == 0 && 8 * c < H) a.scale[t * groups + c / 16] = __fdiv_rn(m, kE4m3Max);
            }
        }
        uint32_t w[K][2];
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float* p = s + 8 * k + 4 * i;
                w[k][i] = uint32_t(e4m3_pair(__fmul_rn(p[0], inv[k]), __fmul_rn(p[1], inv[k]))) |
                          uint32_t(e4m3_pair(__fmul_rn(p[2], inv[k]), __fmul_rn(p[3], inv[k]))) << 16;
            }
        if constexpr (VEC) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const uint32_t c = 8 * (j + k * nt);
                if (c < H) __stcs(reinterpret_cast<uint2*>(y + c), make_uint2(w[k][0], w[k][1]));
            }
        } else {
            publish_edges<2, K>(edge, w);
            if (nt > 32) __syncthreads();
            store_unaligned<1, K>(reinterpret_cast<char*>(y), H, w, edge);
        }
    }
}

// Forward: block (nt, rows); rows > 1 only with nt = 32 (a warp per row, no barrier).
template <int DT, int K, bool VEC, int OUT>
__global__ void __launch_bounds__(kMaxThreads, K <= 2 ? 2 : 1) fwd_kernel(const FwdArgs a) {
    pdl_enter();
    __shared__ Fold shared[2];
    __shared__ uint4 edge[VEC ? 1 : 2][VEC ? 1 : kEdges];
    const int64_t t = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    if (t >= a.T) return;
    clear_fold(shared, 2);
    const uint32_t H = a.H, j = threadIdx.x;
    F2 s[4 * K];
    uint32_t total[K][4];
    {
        Words<4> x[K], r[K];
        load_words<K, VEC>(Input(a.x, a.x_stride, a.T, H), t, H, x);
        if (a.residual != nullptr) load_words<K, VEC>(Input(a.residual, a.residual_stride, a.T, H), t, H, r);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[4 * k + i] = pair_of<DT>(x[k].w[i]);
        if (a.residual != nullptr) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[4 * k + i] = padd(s[4 * k + i], pair_of<DT>(r[k].w[i]));
            pack_row<DT, K>(s, total);
            if constexpr (VEC) store_aligned<K>(a.total + t * int64_t(H), H, total);
            else publish_edges<4, K>(edge[0], total);
        }
    }
    const float sum = fold(squares<K>(s), shared[0], Add());   // (a barrier, where a row has more than one warp)
    if constexpr (!VEC)
        if (a.residual != nullptr) store_unaligned<2, K>(reinterpret_cast<char*>(a.total + t * int64_t(H)), H, total, edge[0]);
    const float rstd = rstd_of(sum, H, a.eps);
    if (j == 0) a.rstd[t] = rstd;
    F2 w[4 * K];
    load_weight<K, VEC>(a.weight, H, w);
    normalise<K>(s, rstd, w);
    store_y<DT, K, VEC, OUT>(a, t, s, shared[1], edge[VEC ? 0 : 1]);
}

// A chunk of the backward's first pass: adds g * n to acc and gives the
// chunk's part of the sum of u * n.
template <int DT>
__device__ __forceinline__ float backward_terms(const Words<4>& g, const Words<4>& s, F2 rstd, const F2* w, F2* acc) {
    F2 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const F2 gv = pair_of<DT>(g.w[i]), n = pmul(pair_of<DT>(s.w[i]), rstd);
        acc[i] = pfma(gv, n, acc[i]);
        q[i] = pmul(pmul(gv, w[i]), n);
    }
    return chunk_sum(q);
}

// And of the second: grad_x.
template <int DT>
__device__ __forceinline__ void backward_values(const Words<4>& g, const Words<4>& s, const Words<4>& more, bool with_more,
                                                F2 rstd, F2 minus_m, const F2* w, F2* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const F2 n = pmul(pair_of<DT>(s.w[i]), rstd);
        const F2 d = pfma(n, minus_m, pmul(pair_of<DT>(g.w[i]), w[i]));
        v[i] = with_more ? pfma(rstd, d, pair_of<DT>(more.w[i])) : pmul(rstd, d);
    }
}

// A block's sums of grad_weight: to its row of the workspace, whose rows are
// of whole chunks, or (`last`: the only block) to grad_weight itself.
template <int K, bool VEC>
__device__ __forceinline__ void store_partial(float* __restrict__ out, uint32_t H, bool last, const F2 (&acc)[4 * K]) {
    const uint32_t nt = blockDim.x, j = threadIdx.x;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const uint32_t c = 8 * (j + k * nt);
        if (VEC || !last) {
            if (c < H) {
                float4* p = reinterpret_cast<float4*>(out + c);
                const F2* v = acc + 4 * k;
                p[0] = make_float4(f2_lo(v[0]), f2_hi(v[0]), f2_lo(v[1]), f2_hi(v[1]));
                p[1] = make_float4(f2_lo(v[2]), f2_hi(v[2]), f2_lo(v[3]), f2_hi(v[3]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < H) out[c + i] = i & 1 ? f2_hi(acc[4 * k + i / 2]) : f2_lo(acc[4 * k + i / 2]);
        }
    }
}

// Backward: block b takes rows b * rows + y, then steps of gridDim.x * rows
// (rows = blockDim.y > 1 only with nt = 32), writes their grad_x and leaves
// the sum of their g * n in partial[b]; the rows of one (b, y) are added in
// increasing order, then the y in increasing order.
template <int DT, int K, bool VEC>
__global__ void __launch_bounds__(kMaxThreads, 1) bwd_kernel(const BwdArgs a) {
    pdl_enter();
    extern __shared__ __align__(16) float stage[];
    __shared__ Fold shared[2];
    __shared__ uint4 edge[VEC ? 1 : 2][VEC ? 1 : kEdges];
    const uint32_t H = a.H, j = threadIdx.x, rows = blockDim.y;
    clear_fold(shared, 2);
    const int64_t step = int64_t(gridDim.x) * rows;
    const Input in_s(a.s, a.s_stride, a.T, H), in_g(a.g, a.g_stride, a.T, H), in_t(a.grad_total, H, a.T, H);
    F2 acc[4 * K];
#pragma unroll
    for (int i = 0; i < 4 * K; ++i) acc[i] = f2(0.0f, 0.0f);
    int turn = 0;
    for (int64_t t = int64_t(blockIdx.x) * rows + threadIdx.y; t < a.T; t += step, turn ^= 1) {
        Words<4> g[K], n[K], more[K];
        load_words<K, VEC>(in_s, t, H, n);
        load_words<K, VEC>(in_g, t, H, g);
        if (a.grad_total != nullptr) load_words<K, VEC>(in_t, t, H, more);
        const float r1 = __ldg(a.rstd + t);
        const F2 rstd = f2(r1, r1);
        F2 w[4 * K];
        load_weight<K, VEC>(a.weight, H, w);
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) sum = __fadd_rn(sum, backward_terms<DT>(g[k], n[k], rstd, w + 4 * k, acc + 4 * k));
        const float m = -__fdiv_rn(fold(sum, shared[turn], Add()), float(H));
        F2 v[4 * K];
#pragma unroll
        for (int k = 0; k < K; ++k)
            backward_values<DT>(g[k], n[k], more[k], a.grad_total != nullptr, rstd, f2(m, m), w + 4 * k, v + 4 * k);
        store_row<DT, K, VEC>(a.grad_x + t * int64_t(H), H, v, edge[VEC ? 0 : turn]);
    }
    if (rows > 1) {   // the warps of a block one after the other, in shared memory
        for (uint32_t y = 0; y < rows; ++y) {
            if (threadIdx.y == y) {
#pragma unroll
                for (int i = 0; i < 4 * K; ++i) {
                    F2* at = reinterpret_cast<F2*>(stage) + j + i * 32;
                    *at = y == 0 ? acc[i] : padd(*at, acc[i]);
                }
            }
            __syncthreads();
        }
        if (threadIdx.y != 0) return;
#pragma unroll
        for (int i = 0; i < 4 * K; ++i) acc[i] = reinterpret_cast<const F2*>(stage)[j + i * 32];
    }
    store_partial<K, VEC>(a.partial + int64_t(blockIdx.x) * a.pitch, H, gridDim.x == 1, acc);
}

// The ring of a block: kept rows of `arrays` buffers, bulk-copied by thread 0.
// Stage i of the ring holds the block's rows i, i + stages, ...; its buffers
// lie one after the other.  A stage is free again after the barrier inside
// the row's sum: by then every thread has its values in registers.
struct RingRows {
    const uint16_t* from[3];
    int64_t stride[3];
    uint32_t arrays;
};

__device__ __forceinline__ void ring_copy(char* stage, const RingRows& r, int64_t t, uint32_t bytes, uint64_t* full) {
    mbar_arrive_expect_tx(full, r.arrays * bytes);
    for (uint32_t i = 0; i < r.arrays; ++i) bulk_copy_g2s(stage + i * bytes, r.from[i] + t * r.stride[i], bytes, full);
}

// Thread 0's end after a wait that ran out: records it and waits (again
// bounded) for the copies in flight.
static __device__ __noinline__ void ring_late(uint64_t* full, uint32_t issued, uint32_t stages, unsigned int* timeouts) {
    *timeouts = 1u;
    for (uint32_t i = issued > stages ? issued - stages : 0; i < issued; ++i) mbar_wait(full + i % stages, (i / stages) & 1);
}

template <int DT, int K>
__device__ __forceinline__ void stage_words(const char* row, uint32_t H, Words<4> (&w)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const uint32_t c = 8 * (threadIdx.x + k * blockDim.x);
        const uint4 v = c < H ? *reinterpret_cast<const uint4*>(row + 2 * c) : make_uint4(0, 0, 0, 0);
        w[k].w[0] = v.x, w[k].w[1] = v.y, w[k].w[2] = v.z, w[k].w[3] = v.w;
    }
}

constexpr uint32_t kRingStages = 4;   // at most

template <int DT, int K, int OUT, int MAXT>
__global__ void __launch_bounds__(MAXT, K == 2 ? 2 : 1)
fwd_ring_kernel(const FwdArgs a, const RingRows r, uint32_t stages) {
    extern __shared__ __align__(16) char ring[];
    __shared__ Fold shared[2][2];
    __shared__ uint64_t full[kRingStages];
    __shared__ volatile int late;   // a wait ran out: no further copy, no further wait
    const uint32_t H = a.H, j = threadIdx.x, bytes = 2 * H;
    if (j == 0) {
        for (uint32_t s = 0; s < stages; ++s) mbar_init(full + s, 1);
        mbar_init_fence();
        late = 0;
    }
    clear_fold(shared[0], 4);
    __syncthreads();
    pdl_enter();
    const int64_t step = gridDim.x;
    uint32_t issued = 0;   // of thread 0
    if (j == 0)
        for (; issued < stages && blockIdx.x + issued * step < a.T; ++issued)
            ring_copy(ring + issued * r.arrays * bytes, r, blockIdx.x + issued * step, bytes, full + issued);
    F2 w[4 * K];
    load_weight<K, true>(a.weight, H, w);
    uint32_t stage = 0, parity = 0;
    int turn = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += step, turn ^= 1) {
        if (!late && !mbar_wait_fast(full + stage, parity)) late = 1;
        const char* row = ring + stage * r.arrays * bytes;
        Words<4> raw[K];
        F2 s[4 * K];
        stage_words<DT, K>(row, H, raw);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[4 * k + i] = pair_of<DT>(raw[k].w[i]);
        if (r.arrays > 1) {
            stage_words<DT, K>(row + bytes, H, raw);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[4 * k + i] = padd(s[4 * k + i], pair_of<DT>(raw[k].w[i]));
            store_row<DT, K, true>(a.total + t * int64_t(H), H, s, nullptr);
        }
        const float sum = fold(squares<K>(s), shared[turn][0], Add());
        if (j == 0 && t + stages * step < a.T && !late) {
            fence_proxy_async_shared();
            ring_copy(ring + stage * r.arrays * bytes, r, t + stages * step, bytes, full + stage);
            ++issued;
        }
        if (++stage == stages) stage = 0, parity ^= 1;
        const float rstd = rstd_of(sum, H, a.eps);
        if (j == 0) a.rstd[t] = rstd;
        normalise<K>(s, rstd, w);
        store_y<DT, K, true, OUT>(a, t, s, shared[turn][1], nullptr);
    }
    if (j == 0 && late) ring_late(full, issued, stages, a.timeouts);
}

template <int DT, int K>
__global__ void __launch_bounds__(kMaxThreads, 1)
bwd_ring_kernel(const BwdArgs a, const RingRows r, uint32_t stages) {
    extern __shared__ __align__(16) char ring[];
    __shared__ Fold shared[2];
    __shared__ uint64_t full[kRingStages];
    __shared__ volatile int late;   // a wait ran out: no further copy, no further wait
    const uint32_t H = a.H, j = threadIdx.x, bytes = 2 * H;
    if (j == 0) {
        for (uint32_t s = 0; s < stages; ++s) mbar_init(full + s, 1);
        mbar_init_fence();
        late = 0;
    }
    clear_fold(shared, 2);
    __syncthreads();
    pdl_enter();
    const int64_t step = gridDim.x;
    uint32_t issued = 0;   // of thread 0
    if (j == 0)
        for (; issued < stages && blockIdx.x + issued * step < a.T; ++issued)
            ring_copy(ring + issued * r.arrays * bytes, r, blockIdx.x + issued * step, bytes, full + issued);
    F2 w[4 * K], acc[4 * K];
    load_weight<K, true>(a.weight, H, w);
#pragma unroll
    for (int i = 0; i < 4 * K; ++i) acc[i] = f2(0.0f, 0.0f);
    uint32_t stage = 0, parity = 0;
    int turn = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += step, turn ^= 1) {
        const float r1 = __ldg(a.rstd + t);
        const F2 rstd = f2(r1, r1);
        if (!late && !mbar_wait_fast(full + stage, parity)) late = 1;
        const char* row = ring + stage * r.arrays * bytes;
        Words<4> g[K], n[K], more[K];
        stage_words<DT, K>(row, H, g);
        stage_words<DT, K>(row + bytes, H, n);
        if (r.arrays > 2) stage_words<DT, K>(row + 2 * bytes, H, more);
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) sum = __fadd_rn(sum, backward_terms<DT>(g[k], n[k], rstd, w + 4 * k, acc + 4 * k));
        const float m = -__fdiv_rn(fold(sum, shared[turn], Add()), float(H));
        if (j == 0 && t + stages * step < a.T && !late) {
            fence_proxy_async_shared();
            ring_copy(ring + stage * r.arrays * bytes, r, t + stages * step, bytes, full + stage);
            ++issued;
        }
        if (++stage == stages) stage = 0, parity ^= 1;
        F2 v[4 * K];
#pragma unroll
        for (int k = 0; k < K; ++k) backward_values<DT>(g[k], n[k], more[k], r.arrays > 2, rstd, f2(m, m), w + 4 * k, v + 4 * k);
        store_row<DT, K, true>(a.grad_x + t * int64_t(H), H, v, nullptr);
    }
    store_partial<K, true>(a.partial + int64_t(blockIdx.x) * a.pitch, H, false, acc);
    if (j == 0 && late) ring_late(full, issued, stages, a.timeouts);
}

// Column sums of partial [P,H] (row pitch `pitch`): a block takes 32 columns,
// 8 threads with four each in 128 groups; group y adds the rows y, y + 128, ...
// in increasing order, then a lane adds four groups and the lanes fold at
// distance 16, 8, 4, 2, 1.  (The rows' latency is what it waits for: with 32
// groups the norm's backward took 2.3 us more.)  VEC: pitch % 4 == 0 and a 16-byte aligned
// partial.  Also the bias gradient's last step.
constexpr int kColGroups = 128;

template <bool VEC>
static __global__ void __launch_bounds__(8 * kColGroups)
column_sum_kernel(const float* __restrict__ partial, float* __restrict__ out, uint32_t P, uint32_t H, uint32_t pitch) {
    pdl_enter();
    __shared__ float part[32][kColGroups + 1];
    const uint32_t x = threadIdx.x % 8, y = threadIdx.x / 8, c = blockIdx.x * 32 + 4 * x;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < H)
#pragma unroll 4
        for (uint32_t p = y; p < P; p += kColGroups) {
            const float* row = partial + uint64_t(p) * pitch + c;
            if constexpr (VEC) {
                const float4 v = *reinterpret_cast<const float4*>(row);
                acc[0] = __fadd_rn(acc[0], v.x), acc[1] = __fadd_rn(acc[1], v.y);
                acc[2] = __fadd_rn(acc[2], v.z), acc[3] = __fadd_rn(acc[3], v.w);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + i < H) acc[i] = __fadd_rn(acc[i], row[i]);
            }
        }
#pragma unroll
    for (int i = 0; i < 4; ++i) part[4 * x + i][y] = acc[i];
    __syncthreads();
    {
        const uint32_t lane = threadIdx.x & 31u, column = threadIdx.x / 32;   // a warp for each
        const float* g = &part[column][4 * lane];
        float v = __fadd_rn(__fadd_rn(g[0], g[1]), __fadd_rn(g[2], g[3]));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
        if (lane == 0 && blockIdx.x * 32 + column < H) out[blockIdx.x * 32 + column] = v;
    }
}

}  // namespace norm
}  // namespace mhc
