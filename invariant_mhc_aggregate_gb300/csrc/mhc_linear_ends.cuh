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
// gated: of each 32 lanes, the first 16 are values f of the gate and the
// others the same f of the up projection, so one exchange within the warp
// brings a pair together and every value's activation is evaluated once.  A
// row's stores are 32 contiguous bytes.
// --------------------------------------------------------------------------

// The row of w [2 F, I] (the column of z) that lane `index` of the tiles
// holds; ok: there is one.
__device__ __forceinline__ int64_t gated_column(int64_t half, int64_t index, bool& ok) {
    const int64_t f = (index >> 5) * 16 + (index & 15);
    ok = f < half;
    return index & 16 ? half + f : f;
}

template <int OUT, int C, bool ALL>
__device__ __forceinline__ void emit_gated(const TileArgs& a, bool n_ok, int64_t n, uint32_t m0, uint32_t step, uint32_t rows,
                                           float (&v)[C], float bias, float col_scale) {
    const Epilogue& e = a.e;
    const bool up = (threadIdx.x & 16) != 0;
    const int64_t half = a.end.half, f = up ? n - half : n;
    auto there = [&](uint32_t m) { return ALL || (n_ok && m < rows); };
    if (e.row_scale != nullptr) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (there(m0 + c * step)) v[c] = __fmul_rn(__fmul_rn(v[c], __ldg(e.row_scale + m0 + c * step)), col_scale);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = __fadd_rn(v[c], bias);
    if (e.preact != nullptr) {
        uint16_t* p = e.preact + int64_t(m0) * (2 * half) + n;
#pragma unroll
        for (int c = 0; c < C; ++c, p += step * (2 * half))
            if (there(m0 + c * step)) *p = Elem<OUT>::cvt(v[c]);
    }
    // the gate's lane takes the first half of the rows, the other lane the second
    float gate[C / 2], other[C / 2];
#pragma unroll
    for (int c = 0; c < C / 2; ++c) {
        const float mine = up ? v[C / 2 + c] : v[c], theirs = __shfl_xor_sync(0xFFFFFFFFu, up ? v[c] : v[C / 2 + c], 16);
        gate[c] = up ? theirs : mine;
        other[c] = up ? mine : theirs;
    }
    switch (e.act) {
        case kActRelu:
#pragma unroll
            for (int c = 0; c < C / 2; ++c) gate[c] = activation<kActRelu>(gate[c]);
            break;
        case kActSilu:
#pragma unroll
            for (int c = 0; c < C / 2; ++c) gate[c] = activation<kActSilu>(gate[c]);
            break;
        case kActGelu:
#pragma unroll
            for (int c = 0; c < C / 2; ++c) gate[c] = activation<kActGelu>(gate[c]);
            break;
        default: break;
    }
    const uint32_t first = m0 + (up ? C / 2 * step : 0);
    uint16_t* p = e.y + int64_t(first) * half + f;
#pragma unroll
    for (int c = 0; c < C / 2; ++c, p += step * half)
        if (there(first + c * step)) *p = Elem<OUT>::cvt(__fmul_rn(gate[c], other[c]));
}

// --------------------------------------------------------------------------
// sums: a product in pieces of K, added up in FP32; the last piece's sum is
// scaled and rounded once
// --------------------------------------------------------------------------
template <int OUT, int C, bool ALL>
__device__ __forceinline__ void emit_sum(const TileArgs& a, bool n_ok, int64_t n, uint32_t m0, uint32_t step, uint32_t rows,
                                         float (&v)[C]) {
    const int64_t at = int64_t(m0) * a.N + n, stride = int64_t(step) * a.N;
    auto there = [&](int c) { return ALL || (n_ok && m0 + c * step < rows); };
    if (a.end.sum_in != nullptr) {
        const float* p = a.end.sum_in + at;
        float w[C];
#pragma unroll
        for (int c = 0; c < C; ++c) w[c] = there(c) ? __ldcs(p + c * stride) : 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = __fadd_rn(w[c], v[c]);
    }
    if (a.end.sum_out != nullptr) {
        float* p = a.end.sum_out + at;
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (there(c)) p[c * stride] = v[c];
    } else {
        const float factor = __ldg(a.end.factor);
        uint16_t* p = a.e.y + at;
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (there(c)) p[c * stride] = Elem<OUT>::cvt(__fmul_rn(v[c], factor));
    }
}

// --------------------------------------------------------------------------
// the gradient of a cross entropy's logits, d = spread exp(z - lse) less the
// target's gradient, from the logits' sums z.  It is rounded to the storage
// type since both products that read it take 16-bit operands.
// --------------------------------------------------------------------------
template <int OUT, int C, bool ALL>
__device__ __forceinline__ void emit_prob(const TileArgs& a, bool n_ok, int64_t n, uint32_t m0, uint32_t step, uint32_t rows,
                                          float (&v)[C]) {
    const int32_t entry = a.end.first + int32_t(n);
    uint16_t* p = a.e.y + int64_t(m0) * a.end.pitch + n;
    const int64_t stride = int64_t(step) * a.end.pitch;
#pragma unroll
    for (int c = 0; c < C; ++c, p += stride) {
        const bool there = ALL || (n_ok && m0 + c * step < rows);
        if (there) {
            const float4 t = __ldg(reinterpret_cast<const float4*>(a.end.tokens) + m0 + c * step);
            // (a token without a gradient has none whatever its logits are)
            float d = t.y == 0.0f ? 0.0f : __fmul_rn(exp_fast(__fsub_rn(v[c], t.x)), t.y);
            if (__float_as_int(t.w) == entry) d = __fsub_rn(d, t.z);
            *p = Elem<OUT>::cvt(d);
        }
    }
}

template <int END, int OUT, int C, bool ALL>
__device__ __forceinline__ void emit_of(const TileArgs& a, bool n_ok, int64_t n, uint32_t m0, uint32_t step, uint32_t rows,
                                        float (&v)[C], float bias, float col_scale) {
    if constexpr (END == kEndGated) emit_gated<OUT, C, ALL>(a, n_ok, n, m0, step, rows, v, bias, col_scale);
    if constexpr (END == kEndSum) emit_sum<OUT, C, ALL>(a, n_ok, n, m0, step, rows, v);
    if constexpr (END == kEndProb) emit_prob<OUT, C, ALL>(a, n_ok, n, m0, step, rows, v);
}

// One chunk by itself (split_kernel).
template <int END, int OUT, int C>
__device__ __forceinline__ void emit_end(const TileArgs& a, bool n_ok, int64_t n, uint32_t m0, uint32_t step, uint32_t rows,
                                         float (&v)[C], float bias, float col_scale) {
    if (__all_sync(0xFFFFFFFFu, n_ok) && m0 + (C - 1) * step < rows)
        emit_of<END, OUT, C, true>(a, n_ok, n, m0, step, rows, v, bias, col_scale);
    else
        emit_of<END, OUT, C, false>(a, n_ok, n, m0, step, rows, v, bias, col_scale);
}

// A warp's `mine` columns of a finished tile, from tensor memory at `from`
// (pair_kernel); give_back after the last read of tensor memory.
template <int END, int OUT, bool ALL, typename GiveBack>
__device__ __forceinline__ void end_columns(const TileArgs& a, uint32_t from, uint32_t mine, uint32_t m0, int64_t col, bool n_ok,
                                            float bias, float cs, GiveBack give_back) {
    constexpr int C = 8;
    float next[C];
    umma::tmem_ld(from, next);
#pragma unroll 1
    for (uint32_t c = 0; c < mine; c += C) {
        umma::tmem_wait_ld(next);
        float v[C];
#pragma unroll
        for (int k = 0; k < C; ++k) v[k] = next[k];
        if (c + C < mine) umma::tmem_ld(from + c + C, next);
        else give_back();
        emit_of<END, OUT, C, ALL>(a, n_ok, col, m0 + c, 1, a.rows, v, bias, cs);
    }
}

template <int END, int OUT, typename GiveBack>
__device__ __forceinline__ void end_tile(const TileArgs& a, uint32_t from, uint32_t mine, uint32_t m0, int64_t col, bool n_ok,
                                         float bias, float cs, GiveBack give_back) {
    if (__all_sync(0xFFFFFFFFu, n_ok) && m0 + mine <= a.rows)
        end_columns<END, OUT, true>(a, from, mine, m0, col, n_ok, bias, cs, give_back);
    else
        end_columns<END, OUT, false>(a, from, mine, m0, col, n_ok, bias, cs, give_back);
}

// --------------------------------------------------------------------------
// cross entropy: the logits' lanes are tokens and their columns entries of
// the vocabulary, so that a thread takes the maximum and the sum of
// exponentials of its `mine` (32 or 64) entries in registers; one such pair a
// group and token goes to memory, 1/16 or 1/32 of the logits' bytes in 16 bits.
// --------------------------------------------------------------------------

// exp(x - ref(x)) needs a finite reference: an infinite maximum has 0.
__device__ __forceinline__ float reference(float top) { return fabsf(top) < INFINITY ? top : 0.0f; }

// (top, sum) and another group's together.
__device__ __forceinline__ void join_groups(float& top, float& sum, float top2, float sum2) {
    const float most = fmaxf(top, top2), ref = reference(most);
    sum = __fadd_rn(__fmul_rn(sum, exp_fast(__fsub_rn(top, ref))), __fmul_rn(sum2, exp_fast(__fsub_rn(top2, ref))));
    top = most;
}

// The longest run of blocks of K that one accumulator sums: the tensor cores
// cut off each addition's last bits, so a logit is short by about half a unit
// of the last place for each 16 products.  Runs are added up in registers,
// rounded to nearest: K = 7168 in one run, lse is 3.9e-6 off (in norm, against
// 64 bits), in runs of 16 blocks 6e-7, FP32 sums of the plain form's 8e-7.
constexpr uint32_t kEntropyRun = 16;
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

// The group of the thread's logits v.
__device__ __forceinline__ void entropy_tile(const TileArgs& a, uint32_t mine, uint32_t m0, int64_t t, bool ok,
                                             float (&v)[kEntropyMost / 8][8]) {
    constexpr int kRun = 32;
    const int64_t target = ok ? __ldg(a.end.target + t) : -1;
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int c = 0; c < kEntropyMost; c += kRun) {
        if (uint32_t(c) >= mine) break;
        const uint32_t first = m0 + c;
        float(*q)[8] = v + c / 8;
        if (first + kRun > a.rows) {   // (the same for the whole warp)
#pragma unroll
            for (int i = 0; i < kRun; ++i)
                if (first + i >= a.rows) q[i / 8][i % 8] = -INFINITY;
        }
        const int64_t rel = target - int64_t(first);
        if (__any_sync(0xFFFFFFFFu, rel >= 0 && rel < kRun)) {
#pragma unroll
            for (int i = 0; i < kRun; ++i)
                if (rel == i) a.end.at[t] = q[i / 8][i % 8];
        }
        float most[8], part[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) most[j] = fmaxf(fmaxf(q[0][j], q[1][j]), fmaxf(q[2][j], q[3][j]));
#pragma unroll
        for (int s = 4; s > 0; s >>= 1)
#pragma unroll
            for (int j = 0; j < s; ++j) most[j] = fmaxf(most[j], most[j + s]);
        const float ref = reference(most[0]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = exp_fast(__fsub_rn(q[i][j], ref));
            part[j] = __fadd_rn(__fadd_rn(w[0], w[1]), __fadd_rn(w[2], w[3]));
        }
#pragma unroll
        for (int s = 4; s > 0; s >>= 1)
#pragma unroll
            for (int j = 0; j < s; ++j) part[j] = __fadd_rn(part[j], part[j + s]);
        if (c == 0) top = most[0], sum = part[0];
        else join_groups(top, sum, most[0], part[0]);
    }
    if (ok && m0 < a.rows) a.end.partial[int64_t(m0 / mine) * a.N + t] = make_float2(top, sum);
}

}  // namespace linear
}  // namespace mhc
