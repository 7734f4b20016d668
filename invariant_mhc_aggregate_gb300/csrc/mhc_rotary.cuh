// Rotary positions (sm_103a): the first R values of every head of a token are
// rotated in pairs by position * frequency, the rest copied.  Definitions in
// mhc_layer.h.
//
// HBM-bound: each value is read and written once.  A thread owns one unit of
// a head row for a run of heads of one token: in the half layout two pieces of
// W values (of the rotated part's two halves, which pair with each other, or
// of the rest's), interleaved one piece of W values (W/2 pairs, or of the
// rest).  Rotated and copied units take the same loads and stores, so that a
// warp that holds both issues them together.  The thread computes its angles'
// cosines and sines once, under its first loads, and reuses them for all its
// heads: the trigonometry is shared without shared memory or a barrier.  T =
// 32768, 40 heads of 128 values, 64 of them rotated: 97.3 us, the copy
// bandwidth (139 us with the trigonometry's library functions, single values
// in place of words and the copied values in a branch of their own).
//
// The angle is the exact product p * f of the position and the FP32 frequency
// (the product and its rounding error, two FP32 numbers; positions past 2^24
// in two parts), reduced by the nearest multiple of 2 pi with 2 pi held in two
// FP32 numbers (Cody and Waite's reduction, with fused multiply-adds): the
// error stays near 1e-6 for positions up to millions, where the FP32 product
// alone would be off by p * 2^-24.
#pragma once

#include "fastdiv.cuh"
#include "mhc_device.cuh"

namespace mhc {
namespace rotary {

struct Args {
    const uint16_t* x;
    uint16_t* out;
    const int64_t* positions;
    const float* frequencies;
    int64_t x_token, x_head, out_token, out_head;
    uint64_t work;            // threads with work: T * runs * units
    uint32_t heads, D, R;
    uint32_t lead, gap;       // two-piece units: the rotated unit u's pieces start at u * lead and u * lead + gap
    uint32_t copy_gap;        // and the copied unit u's at R + u * W and R + u * W + copy_gap (if still before D)
    uint32_t run;             // heads of one thread
    uint32_t rot_units;       // units of the rotated part of a head
    FastDivU32 by_units, by_runs;
    float magnitude;          // with the sign of the sines in `sine_sign`
    float sine_sign;
};

constexpr float kTwoPiHigh = 0x1.921fb6p+2f;      // RN(2 pi)
constexpr float kTwoPiLow = -0x1.777a5cp-23f;     // RN(2 pi - kTwoPiHigh)
constexpr float kInvTwoPi = 0x1.45f306p-3f;       // RN(1 / (2 pi))

// position = high + low (low is 0 up to 2^24).  The reduced angle is within
// pi, where the hardware's sine and cosine are within 2^-21 of the exact ones,
// far below the rounding of the result to 11 bits or fewer.
__device__ __forceinline__ void cos_sin(float high, float low, float f, float& c, float& s) {
    const float p = __fmul_rn(high, f);
    const float e = __fmaf_rn(low, f, __fmaf_rn(high, f, -p));
    const float n = rintf(__fmul_rn(p, kInvTwoPi));
    const float r = __fadd_rn(__fmaf_rn(-n, kTwoPiLow, __fmaf_rn(-n, kTwoPiHigh, p)), e);
    s = __sinf(r);
    c = __cosf(r);
}

// W values in 32-bit words, moved with one access (W = 8, 4, 2, 1: 16, 8, 4,
// 2 bytes).  Not the read-only path: x may be out itself.
template <int W>
struct Piece {
    uint32_t w[(W + 1) / 2];
};

template <int W>
__device__ __forceinline__ Piece<W> load(const uint16_t* p) {
    Piece<W> r;
    if constexpr (W == 8) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
        r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
    } else if constexpr (W == 4) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
        r.w[0] = v.x, r.w[1] = v.y;
    } else if constexpr (W == 2) {
        r.w[0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
    } else {
        r.w[0] = __ldcs(p);
    }
    return r;
}

template <int W>
__device__ __forceinline__ void store(uint16_t* p, const Piece<W>& r) {
    if constexpr (W == 8)
        __stcs(reinterpret_cast<uint4*>(p), make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]));
    else if constexpr (W == 4)
        __stcs(reinterpret_cast<uint2*>(p), make_uint2(r.w[0], r.w[1]));
    else if constexpr (W == 2)
        __stcs(reinterpret_cast<uint32_t*>(p), r.w[0]);
    else
        __stcs(p, uint16_t(r.w[0]));
}

// (a, b) -> (a c - b s, b c + a s), a product of each in a fused multiply-add
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
    const float x = a;
    a = __fmaf_rn(x, c, -__fmul_rn(b, s));
    b = __fmaf_rn(b, c, __fmul_rn(x, s));
}

// The pairs of a unit: in the words of one piece, or across two pieces.
template <int DT, int W>
__device__ __forceinline__ void turn_within(Piece<W>& p, const float (&c)[W / 2], const float (&s)[W / 2]) {
#pragma unroll
    for (int k = 0; k < W / 2; ++k) {
        float a = Elem<DT>::lo(p.w[k]), b = Elem<DT>::hi(p.w[k]);
        turn(a, b, c[k], s[k]);
        p.w[k] = Elem<DT>::pack(a, b);
    }
}

template <int DT, int W>
__device__ __forceinline__ void turn_across(Piece<W>& p, Piece<W>& q, const float (&c)[W], const float (&s)[W]) {
    if constexpr (W == 1) {
        float a = Elem<DT>::one(uint16_t(p.w[0])), b = Elem<DT>::one(uint16_t(q.w[0]));
        turn(a, b, c[0], s[0]);
        p.w[0] = Elem<DT>::cvt(a), q.w[0] = Elem<DT>::cvt(b);
    } else {
#pragma unroll
        for (int k = 0; k < W / 2; ++k) {
            float a0 = Elem<DT>::lo(p.w[k]), b0 = Elem<DT>::lo(q.w[k]);
            float a1 = Elem<DT>::hi(p.w[k]), b1 = Elem<DT>::hi(q.w[k]);
            turn(a0, b0, c[2 * k], s[2 * k]);
            turn(a1, b1, c[2 * k + 1], s[2 * k + 1]);
            p.w[k] = Elem<DT>::pack(a0, a1), q.w[k] = Elem<DT>::pack(b0, b1);
        }
    }
}

constexpr int kThreads = 256;

// INTERLEAVED: a unit is one piece that holds W / 2 whole pairs (W >= 2).
// Otherwise it is two pieces that pair with each other: the two halves' (lead
// = W, gap = R / 2), or the two values of one interleaved pair where nothing
// wider is aligned (W = 1, lead = 2, gap = 1).
template <int DT, int W, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const Args a) {
    pdl_enter();
    constexpr int P = INTERLEAVED ? W / 2 : W;           // pairs of a unit
    constexpr uint32_t kBatch = INTERLEAVED ? 8 : 4;     // heads whose loads are issued before the first store
    const uint64_t i = uint64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= a.work) return;
    const uint32_t rest = fastdiv_u32(uint32_t(i), a.by_units);
    const uint32_t unit = uint32_t(i) - rest * a.by_units.d;
    const uint32_t t = fastdiv_u32(rest, a.by_runs);
    const uint32_t h0 = (rest - t * a.by_runs.d) * a.run;
    const uint32_t h1 = min(h0 + a.run, a.heads);
    const bool rotated = unit < a.rot_units;
    const uint32_t at = rotated ? unit * (INTERLEAVED ? W : a.lead) : a.R + (unit - a.rot_units) * W;
    const uint32_t gap = rotated ? a.gap : a.copy_gap;
    const bool second = !INTERLEAVED && at + gap < a.D;
    const uint16_t* x = a.x + int64_t(t) * a.x_token + int64_t(h0) * a.x_head + at;
    uint16_t* out = a.out + int64_t(t) * a.out_token + int64_t(h0) * a.out_head + at;
    float c[P], s[P];
    for (uint32_t h = h0; h < h1; h += kBatch) {
        const uint32_t n = min(kBatch, h1 - h);
        Piece<W> u[kBatch], v[INTERLEAVED ? 1 : kBatch];
#pragma unroll
        for (uint32_t b = 0; b < kBatch; ++b)
            if (b < n) {
                u[b] = load<W>(x + b * a.x_head);
                if constexpr (!INTERLEAVED)
                    if (second) v[b] = load<W>(x + b * a.x_head + gap);
            }
        if (h == h0 && rotated) {
            const int64_t position = __ldg(a.positions + t);
            const float high = __ll2float_rn(position), low = __ll2float_rn(position - __float2ll_rn(high));
#pragma unroll
            for (int k = 0; k < P; ++k) {
                cos_sin(high, low, __ldg(a.frequencies + unit * P + k), c[k], s[k]);
                c[k] = __fmul_rn(c[k], a.magnitude);
                s[k] = __fmul_rn(s[k], a.sine_sign * a.magnitude);
            }
        }
#pragma unroll
        for (uint32_t b = 0; b < kBatch; ++b)
            if (b < n) {
                if (rotated) {
                    if constexpr (INTERLEAVED) turn_within<DT, W>(u[b], c, s);
                    else turn_across<DT, W>(u[b], v[b], c, s);
                }
                store<W>(out + b * a.out_head, u[b]);
                if constexpr (!INTERLEAVED)
                    if (second) store<W>(out + b * a.out_head + gap, v[b]);
            }
        x += kBatch * a.x_head;
        out += kBatch * a.out_head;
    }
}

}  // namespace rotary
}  // namespace mhc
