// What a product ends in beside its own epilogue (mhc_linear.cuh, whose
// kernels call these with sums out of tensor memory: a thread has one lane
// and a chunk of columns, that is, output column n and C output rows).
#pragma once

#include "mhc_linear.cuh"

namespace mhc {
namespace linear {

// The exponential of x by the hardware's power of two (ex2.approx: 2 units of
// the last FP32 place), with results under 2^-126 flushed to 0: beside sums of
// at least 1 and probabilities rounded to 11 bits or fewer they are nothing.
__device__ __forceinline__ float exp_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(__fmul_rn(x, 1.4426950408889634f)));
    return y;
}

// --------------------------------------------------------------------------
// gated: the first half of a tile's lanes is values f of the gate, the second
// half the same f of the up projection (two copies of weight rows as they
// are).  The four warps of a group, which hold the lanes of the same columns,
// put 8 columns of z in shared memory at a time and take it out by pairs: every
// value's activation is evaluated once, and a warp stores 64 contiguous bytes.
// T = 4096, 7168 -> 2 x 14336 870 to 910 us in short runs (1850 to 1940 TFLOP/s; the
// tensor cores), 998 in calls one after the other; with z 4096 -> 2 x 7168 261 to 301
// and 296 us; E4M3 454 and 461 to 469 us.  (Gate and up rows in turn on the
// lanes by small boxes of a 3-D map, paired by shuffles, were as fast.)
// --------------------------------------------------------------------------
constexpr uint32_t kExchange = 8 * kLanesP * 4;   // bytes of a group

struct Gated {
    float* z;             // the group's [8][kLanesP]
    uint32_t barrier;     // the group's
    uint32_t lane;        // of the tile
    int64_t f0;           // the tile's first f
};

// The thread's place; n becomes the row of w (the column of z) that its lane
// holds, n_ok whether there is one.
__device__ __forceinline__ Gated gated_place(const TileArgs& a, char* stages, uint32_t group, uint32_t lane, int64_t f0, int64_t& n,
                                             bool& n_ok) {
    const uint32_t half = a.lanes / 2;
    const int64_t f = f0 + (lane < half ? lane : lane - half);
    n = lane < half ? f : a.end.half + f;
    n_ok = lane < a.lanes && f < a.end.half;
    return {reinterpret_cast<float*>(stages + a.end.exchange + group * kExchange), 1 + group, lane, f0};
}

template <int ACT>
__device__ __forceinline__ void gate_all(float (&v)[4]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = activation<ACT>(v[c]);
}

// 8 columns of z (output rows m0, m0 + step, ...), by the whole group.
template <int OUT>
__device__ __forceinline__ void gated_chunk(const TileArgs& a, const Gated& g, bool n_ok, int64_t n, uint32_t m0, uint32_t step,
                                            uint32_t rows, float (&v)[8], float bias, float col_scale) {
    const Epilogue& e = a.e;
    const int64_t half = a.end.half;
    if (e.row_scale != nullptr) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (m0 + c * step < rows) v[c] = __fmul_rn(__fmul_rn(v[c], __ldg(e.row_scale + m0 + c * step)), col_scale);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = __fadd_rn(v[c], bias);
    if (e.preact != nullptr) {
        uint16_t* p = e.preact + int64_t(m0) * (2 * half) + n;
#pragma unroll
        for (int c = 0; c < 8; ++c, p += step * (2 * half))
            if (n_ok && m0 + c * step < rows) *p = Elem<OUT>::cvt(v[c]);
    }
    umma::group_sync(g.barrier, 128);   // the chunk before has been taken out
#pragma unroll
    for (int c = 0; c < 8; ++c) g.z[c * kLanesP + g.lane] = v[c];
    umma::group_sync(g.barrier, 128);
    // the first two warps take columns 0 .. 3 of 64 values f, the other two 4 .. 7
    const uint32_t i = g.lane & 63, c0 = g.lane >> 6 << 2;
    const float* z = g.z + c0 * kLanesP + i;
    float gate[4], up[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) gate[c] = z[c * kLanesP], up[c] = z[c * kLanesP + a.lanes / 2];
    switch (e.act) {
        case kActRelu: gate_all<kActRelu>(gate); break;
        case kActSilu: gate_all<kActSilu>(gate); break;
        case kActGelu: gate_all<kActGelu>(gate); break;
        default: break;
    }
    if (i < a.lanes / 2 && g.f0 + i < half) {
        uint32_t m = m0 + c0 * step;
        uint16_t* p = e.y + int64_t(m) * half + g.f0 + i;
#pragma unroll
        for (int c = 0; c < 4; ++c, m += step, p += step * half)
            if (m < rows) *p = Elem<OUT>::cvt(__fmul_rn(gate[c], up[c]));
    }
    __syncwarp();
}

// A warp's `mine` columns of a finished tile, from tensor memory at `from`
// (pair_kernel); give_back after the last read of tensor memory.
template <int OUT, typename GiveBack>
__device__ __forceinline__ void gated_tile(const TileArgs& a, const Gated& g, uint32_t from, uint32_t mine, uint32_t m0, int64_t col,
                                           bool n_ok, float bias, float cs, GiveBack give_back) {
    float next[8];
    umma::tmem_ld(from, next);
#pragma unroll 1
    for (uint32_t c = 0; c < mine; c += 8) {
        umma::tmem_wait_ld(next);
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = next[k];
        if (c + 8 < mine) umma::tmem_ld(from + c + 8, next);
        else give_back();
        gated_chunk<OUT>(a, g, n_ok, col, m0 + c, 1, a.rows, v, bias, cs);
    }
}

// --------------------------------------------------------------------------
// sums: a product in pieces of K (calls) and parts (tiles of one call), the
// pieces added up in FP32, each part in a buffer of its own; without buffers,
// the only sum is scaled and rounded here
// --------------------------------------------------------------------------
template <int OUT, int C, bool ALL>
__device__ __forceinline__ void emit_sum(const TileArgs& a, bool n_ok, int64_t n, uint32_t m0, uint32_t step, uint32_t rows,
                                         float (&v)[C], uint32_t part) {
    const int64_t at = int64_t(m0) * a.N + n, stride = int64_t(step) * a.N, apart = int64_t(part) * a.rows * a.N;
    auto there = [&](int c) { return ALL || (n_ok && m0 + c * step < rows); };
    if (a.end.sum_in != nullptr) {
        const float* p = a.end.sum_in + apart + at;
        float w[C];
#pragma unroll
        for (int c = 0; c < C; ++c) w[c] = there(c) ? __ldcs(p + c * stride) : 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = __fadd_rn(w[c], v[c]);
    }
    if (a.end.sum_out != nullptr) {
        float* p = a.end.sum_out + apart + at;
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (there(c)) p[c * stride] = v[c];
    } else {
        const float factor = a.end.scale == nullptr ? 1.0f : __ldg(a.end.scale);
        uint16_t* p = a.e.y + at;
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (there(c)) p[c * stride] = Elem<OUT>::cvt(__fmul_rn(v[c], factor));
    }
}

template <int OUT, bool ALL, typename GiveBack>
__device__ __forceinline__ void sum_columns(const TileArgs& a, uint32_t from, uint32_t mine, uint32_t m0, int64_t col, bool n_ok,
                                            uint32_t part, GiveBack give_back) {
    constexpr int C = 8;
    float next[C];
    umma::tmem_ld(from, next);
#pragma unroll 1
    for (uint32_t c = 0; c < mine; c += C) {
        __syncwarp();   // (after stores that some lanes make)
        umma::tmem_wait_ld(next);
        float v[C];
#pragma unroll
        for (int k = 0; k < C; ++k) v[k] = next[k];
        if (c + C < mine) umma::tmem_ld(from + c + C, next);
        else give_back();
        emit_sum<OUT, C, ALL>(a, n_ok, col, m0 + c, 1, a.rows, v, part);
    }
}

// A warp's `mine` columns of a finished tile, from tensor memory at `from`
// (pair_kernel); give_back after the last read of tensor memory.
template <int OUT, typename GiveBack>
__device__ __forceinline__ void sum_tile(const TileArgs& a, uint32_t from, uint32_t mine, uint32_t m0, int64_t col, bool n_ok,
                                         uint32_t part, GiveBack give_back) {
    if (__all_sync(0xFFFFFFFFu, n_ok) && m0 + mine <= a.rows)
        sum_columns<OUT, true>(a, from, mine, m0, col, n_ok, part, give_back);
    else
        sum_columns<OUT, false>(a, from, mine, m0, col, n_ok, part, give_back);
}

// --------------------------------------------------------------------------
// rows: the lanes are the output's rows, so a thread has runs of 16 values of
// one (each fourth run of the tile, its group's) and stores 32 bytes at a time
// where the rows allow it, 1 KB a warp (with the contiguous index on the lanes
// 64 bytes; short K is bound by the stores: the gradients of T = 8 tokens, I =
// 1024, 128000 entries 195 -> 158 us, T = 1024 668 -> 591).
//
// kEndProb: d = s ((g + grad_lse) exp(z - lse) - (at the target) g), from the
// logits' sums z; g is the gradient of the loss, 0 for an ignored token.  It is
// rounded to the storage type since both products that read it take 16-bit
// operands.  A token without a gradient has d = 0 whatever its logits are.
// kEndRow: z by the scale.
// --------------------------------------------------------------------------
struct RowHead {
    float lse = 0.0f, factor = 1.0f, target_grad = 0.0f;
    int64_t at = -1;   // the target's column
};

// The scale s of a call's d.  A mean over tokens gives all of them one g, whose
// rounding to 16 bits would put every target's gradient off by the same part,
// up to half a step (a mean of some 3690 tokens: BF16 gradients 3.0e-3 off in
// norm, so 1.9e-3); s is a power of two over the largest |g|, which leaves such a
// g none.  The power of two brings the largest gradient to 2^13 .. 2^14, so that
// binary16 holds probabilities down to 2^-38 of it.  Without a usable g, s is
// the power of two alone.
struct Scale {
    float by, inverse;
};

// By THREADS threads (from 0 on) over all of the call's tokens.
template <int THREADS>
__device__ __forceinline__ Scale scale_of(const EndArgs& e, int64_t tokens) {
    __shared__ float2 part[THREADS / 32];
    float one = 0.0f, most = 0.0f;   // the largest |g|, |g + grad_lse|
#pragma unroll 4
    for (int64_t t = threadIdx.x; t < tokens; t += THREADS) {
        const int64_t target = __ldg(e.target + t);
        const float g = e.grad_loss != nullptr && target >= 0 && target < e.entries ? __ldg(e.grad_loss + t) : 0.0f;
        const float spread = e.grad_lse == nullptr ? g : __fadd_rn(g, __ldg(e.grad_lse + t));
        one = fmaxf(one, fabsf(g)), most = fmaxf(most, fmaxf(fabsf(g), fabsf(spread)));
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
        one = fmaxf(one, __shfl_xor_sync(0xFFFFFFFFu, one, s));
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, s));
    }
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = make_float2(one, most);
    umma::group_sync(1, THREADS);
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) one = fmaxf(one, part[w].x), most = fmaxf(most, part[w].y);
    const float tiny = 8.6736174e-19f, huge = 1.1529215e18f;   // 2^-60, 2^60: their quotient is finite
    if (!(one >= tiny && one <= huge && most <= huge)) one = 1.0f;
    const float r = __frcp_rn(one), top = __fmul_rn(most, r);
    int power = 0;
    if (top > 0.0f && top < INFINITY) power = min(13 - ilogbf(top), 126);
    return {ldexpf(r, power), ldexpf(one, -power)};
}

// (read while the row's sums are still under way)
template <int END>
__device__ __forceinline__ RowHead row_head(const TileArgs& a, int64_t row, bool ok, float scale) {
    RowHead h;
    if constexpr (END == kEndProb) {
        if (ok) {
            const int64_t target = __ldg(a.end.target + row);
            const float g = a.end.grad_loss == nullptr ? 0.0f : __ldg(a.end.grad_loss + row);
            h.lse = __ldg(a.end.lse + row);
            if (target >= 0 && target < a.end.entries) {
                h.at = target - a.end.first;
                h.target_grad = g;
            }
            h.factor = a.end.grad_lse == nullptr ? h.target_grad : __fadd_rn(h.target_grad, __ldg(a.end.grad_lse + row));
            h.target_grad = __fmul_rn(h.target_grad, scale);
            h.factor = __fmul_rn(h.factor, scale);
        }
    } else if (a.end.scale != nullptr) {
        h.factor = __ldg(a.end.scale);
    }
    return h;
}

template <int END, int OUT, typename GiveBack>
__device__ __forceinline__ void row_tile(const TileArgs& a, const RowHead& h, uint32_t from, uint32_t group, uint32_t m0, int64_t row,
                                         bool ok, GiveBack give_back) {
    constexpr uint32_t C = 16, kStep = 4 * C;
    uint16_t* p = a.e.y + row * a.end.pitch + m0;
    const uint32_t mask = ok ? uint32_t(reinterpret_cast<uintptr_t>(a.e.y) | uintptr_t(a.end.pitch * 2) | (m0 * 2)) & 31u : 31u;
    const bool sectors = mask == 0, halves = (mask & 15u) == 0;   // (columns of a tile begin at multiples of 16)
    float v[2][8];
    umma::tmem_ld(from + group * C, v[0]);
    umma::tmem_ld(from + group * C + 8, v[1]);
#pragma unroll 1
    for (uint32_t c = group * C; c < a.width; c += kStep) {
        __syncwarp();   // (after stores that some lanes make)
        umma::tmem_wait_ld(v[0]);
        umma::tmem_wait_ld(v[1]);
        float x[C];
#pragma unroll
        for (int k = 0; k < int(C); ++k) x[k] = v[k / 8][k % 8];
        if (c + kStep < a.width) {
            umma::tmem_ld(from + c + kStep, v[0]);
            umma::tmem_ld(from + c + kStep + 8, v[1]);
        } else {
            give_back();
        }
        if constexpr (END == kEndProb) {
            const bool some = h.factor != 0.0f;
#pragma unroll
            for (int k = 0; k < int(C); ++k) x[k] = some ? __fmul_rn(exp_fast(__fsub_rn(x[k], h.lse)), h.factor) : 0.0f;
            const int64_t rel = h.at - int64_t(m0 + c);
            if (__any_sync(0xFFFFFFFFu, rel >= 0 && rel < int64_t(C))) {
#pragma unroll
                for (int k = 0; k < int(C); ++k)
                    if (rel == k) x[k] = __fsub_rn(x[k], h.target_grad);
            }
        } else {
#pragma unroll
            for (int k = 0; k < int(C); ++k) x[k] = __fmul_rn(x[k], h.factor);
        }
        uint32_t w[C / 2];
#pragma unroll
        for (int k = 0; k < int(C) / 2; ++k) w[k] = Elem<OUT>::pack(x[2 * k], x[2 * k + 1]);
        uint16_t* q = p + c;
        const bool whole = m0 + c + C <= a.rows;
        if (sectors && whole) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                         :
                         : "l"(q), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                         : "memory");
        } else if (halves && whole) {
            *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(q + 8) = make_uint4(w[4], w[5], w[6], w[7]);
        } else if (ok) {
#pragma unroll
            for (int k = 0; k < int(C); ++k)
                if (m0 + c + k < a.rows) q[k] = uint16_t(w[k / 2] >> (k % 2 * 16));
        }
    }
}

// --------------------------------------------------------------------------
// cross entropy: the logits' lanes are tokens and their columns entries of
// the vocabulary, so that a thread takes the maximum and the sum of
// exponentials of its `mine` (32 or 64) entries in registers; one such pair a
// group (32 or 64 entries) and token goes to memory, 1/8 or 1/16 of the
// logits' bytes in 16 bits.  A unit of 16 entries has a maximum and a sum of its
// own, units are joined in increasing order, so that few_kernel, with the
// vocabulary on the lanes, has the same sums in the same order.  Under the
// multiplications of the next tile: T = 4096, I = 7168, 65536 entries 1.91 to
// 2.05 ms in short runs (1880 to 2010 TFLOP/s), 2.20 in calls one after the
// other, bound by the tensor cores and their power.
// --------------------------------------------------------------------------
constexpr int kEntropyUnit = 16;

// exp(x - ref(x)) needs a finite reference: an infinite maximum has 0.
__device__ __forceinline__ float reference(float top) { return fabsf(top) < INFINITY ? top : 0.0f; }

// (top, sum) and another group's together.
__device__ __forceinline__ void join_groups(float& top, float& sum, float top2, float sum2) {
    const float most = fmaxf(top, top2), ref = reference(most);
    sum = __fadd_rn(__fmul_rn(sum, exp_fast(__fsub_rn(top, ref))), __fmul_rn(sum2, exp_fast(__fsub_rn(top2, ref))));
    top = most;
}

// A unit's maximum and sum of exponentials, of 16 lanes' entries x (-inf past the vocabulary).
__device__ __forceinline__ float2 entropy_unit(float x) {
    float top = x;
#pragma unroll
    for (int s = 8; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, s));
    float sum = exp_fast(__fsub_rn(x, reference(top)));
#pragma unroll
    for (int s = 8; s > 0; s >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xFFFFFFFFu, sum, s));
    return make_float2(top, sum);
}

// The longest run of blocks of K that one accumulator sums: the tensor cores
// cut off each addition's last bits, so a logit is short by about half a unit
// of the last place for each 16 products.  Runs are added up in registers,
// rounded to nearest: K = 7168 in one run, lse is 3.9e-6 off (in norm, against
// 64 bits), in runs of 16 blocks (kEntropyRun) 5e-7, with 32-bit products and
// sums 8e-7; the time is the same.
constexpr int kEntropyMost = 64;   // entries of a thread

// Adds a finished run of `mine` columns, in tensor memory at `from`, to v.
template <bool FIRST>
__device__ __forceinline__ void entropy_add(uint32_t from, uint32_t mine, float (&v)[kEntropyMost / 8][8]) {
#pragma unroll
    for (uint32_t i = 0; i < kEntropyMost / 8; i += 2) {
        if (8 * i >= mine) break;
        float w[2][8];
        umma::tmem_ld(from + 8 * i, w[0]);
        umma::tmem_ld(from + 8 * i + 8, w[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            umma::tmem_wait_ld(w[k]);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i + k][j] = FIRST ? w[k][j] : __fadd_rn(v[i + k][j], w[k][j]);
        }
    }
}

// The groups of the thread's logits v, of token t (ok: there is one).
__device__ __forceinline__ void entropy_tile(const TileArgs& a, uint32_t mine, uint32_t m0, int64_t t, bool ok, int64_t target,
                                             float (&v)[kEntropyMost / 8][8]) {
    if (m0 + mine > a.rows) {   // (the same for the whole warp)
#pragma unroll
        for (int i = 0; i < kEntropyMost; ++i)
            if (m0 + i >= a.rows) v[i / 8][i % 8] = -INFINITY;
    }
    const int64_t rel = target - int64_t(m0);
    if (__any_sync(0xFFFFFFFFu, rel >= 0 && rel < mine)) {
#pragma unroll
        for (int i = 0; i < kEntropyMost; ++i)
            if (rel == i && uint32_t(i) < mine) a.end.at[t] = v[i / 8][i % 8];
    }
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int c = 0; c < kEntropyMost; c += kEntropyUnit) {
        if (uint32_t(c) >= mine) break;
        float(*q)[8] = v + c / 8;
        float most[8], part[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) most[j] = fmaxf(q[0][j], q[1][j]);
#pragma unroll
        for (int s = 4; s > 0; s >>= 1)
#pragma unroll
            for (int j = 0; j < s; ++j) most[j] = fmaxf(most[j], most[j + s]);
        const float ref = reference(most[0]);
#pragma unroll
        for (int j = 0; j < 8; ++j) part[j] = __fadd_rn(exp_fast(__fsub_rn(q[0][j], ref)), exp_fast(__fsub_rn(q[1][j], ref)));
#pragma unroll
        for (int s = 4; s > 0; s >>= 1)
#pragma unroll
            for (int j = 0; j < s; ++j) part[j] = __fadd_rn(part[j], part[j + s]);
        if (c % 32 == 0 && (c == 0 || a.end.group == 32)) top = most[0], sum = part[0];
        else join_groups(top, sum, most[0], part[0]);
        // a group's end
        if (c % 32 == 16 && (c % 64 == 48 || a.end.group == 32)) {
            const uint32_t first = m0 + c + kEntropyUnit - a.end.group;
            if (ok && first < a.rows) a.end.partial[t * a.end.units + first / a.end.group] = make_float2(top, sum);
        }
    }
}

}  // namespace linear
}  // namespace mhc
