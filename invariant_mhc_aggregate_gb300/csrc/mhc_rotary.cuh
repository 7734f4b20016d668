// Rotary positions (sm_103a): the first R values of every head of a token are
// rotated in pairs by position * frequency, the rest copied.  Definitions in
// mhc_layer.h.
//
// HBM-bound: each value is read and written once.  A thread owns one unit of
// a head row for a run of heads of one token: W adjacent pairs (half layout:
// W values of the first half of the rotated part and the W that they pair
// with; interleaved: W/2 pairs in W adjacent values) or, past the rotated
// part, W values to copy.  It computes its angles' cosines and sines once and
// reuses them for all its heads, so the trigonometry is shared without shared
// memory or a barrier.
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
    uint32_t heads, rotated;  // rotated = R
    uint32_t lead, gap;       // two-piece units: unit u's pieces start at u * lead and u * lead + gap
    uint32_t run;             // heads of one thread
    uint32_t rot_units;       // units of the rotated part of a head
    FastDivU32 by_units, by_runs;
    float magnitude;          // with the sign of the sines in `sine_sign`
    float sine_sign;
};

constexpr float kTwoPiHigh = 0x1.921fb6p+2f;      // RN(2 pi)
constexpr float kTwoPiLow = -0x1.777a5cp-23f;     // RN(2 pi - kTwoPiHigh)
constexpr float kInvTwoPi = 0x1.45f306p-3f;       // RN(1 / (2 pi))

__device__ __forceinline__ void cos_sin(int64_t position, float f, float& c, float& s) {
    const float high = __ll2float_rn(position);
    const float low = __ll2float_rn(position - __float2ll_rn(high));
    const float p = __fmul_rn(high, f);
    const float e = __fmaf_rn(low, f, __fmaf_rn(high, f, -p));
    const float n = rintf(__fmul_rn(p, kInvTwoPi));
    const float r = __fadd_rn(__fmaf_rn(-n, kTwoPiLow, __fmaf_rn(-n, kTwoPiHigh, p)), e);
    sincosf(r, &s, &c);
}

template <int W>
struct Piece {
    uint16_t v[W];
};

// W values with one access (W = 8, 4, 2, 1: 16, 8, 4, 2 bytes).  Not the
// read-only path: x may be out itself.
template <int W>
__device__ __forceinline__ Piece<W> load(const uint16_t* p) {
    Piece<W> r;
    if constexpr (W == 8) {
        const uint4 w = __ldcs(reinterpret_cast<const uint4*>(p));
        r.v[0] = uint16_t(w.x), r.v[1] = uint16_t(w.x >> 16), r.v[2] = uint16_t(w.y), r.v[3] = uint16_t(w.y >> 16);
        r.v[4] = uint16_t(w.z), r.v[5] = uint16_t(w.z >> 16), r.v[6] = uint16_t(w.w), r.v[7] = uint16_t(w.w >> 16);
    } else if constexpr (W == 4) {
        const uint2 w = __ldcs(reinterpret_cast<const uint2*>(p));
        r.v[0] = uint16_t(w.x), r.v[1] = uint16_t(w.x >> 16), r.v[2] = uint16_t(w.y), r.v[3] = uint16_t(w.y >> 16);
    } else if constexpr (W == 2) {
        const uint32_t w = __ldcs(reinterpret_cast<const uint32_t*>(p));
        r.v[0] = uint16_t(w), r.v[1] = uint16_t(w >> 16);
    } else {
        r.v[0] = __ldcs(p);
    }
    return r;
}

template <int W>
__device__ __forceinline__ void store(uint16_t* p, const Piece<W>& r) {
    if constexpr (W == 8) {
        Words<4> w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w.w[i] = uint32_t(r.v[2 * i]) | uint32_t(r.v[2 * i + 1]) << 16;
        st_stream<4>(p, w);
    } else if constexpr (W == 4) {
        __stcs(reinterpret_cast<uint2*>(p), make_uint2(uint32_t(r.v[0]) | uint32_t(r.v[1]) << 16,
                                                       uint32_t(r.v[2]) | uint32_t(r.v[3]) << 16));
    } else if constexpr (W == 2) {
        st_stream4(p, uint32_t(r.v[0]) | uint32_t(r.v[1]) << 16);
    } else {
        st_stream2(p, r.v[0]);
    }
}

template <int DT>
__device__ __forceinline__ void turn(uint16_t& a, uint16_t& b, float c, float s) {
    const float x = Elem<DT>::one(a), y = Elem<DT>::one(b);
    a = Elem<DT>::cvt(__fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s)));
    b = Elem<DT>::cvt(__fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s)));
}

constexpr int kThreads = 256;
constexpr uint32_t kBatch = 4;   // heads whose loads are issued before the first store

// INTERLEAVED: a unit is one piece that holds W / 2 whole pairs (W >= 2).
// Otherwise it is two pieces of W values that pair with each other: the two
// halves' (lead = W, gap = R / 2), or the two values of one interleaved pair
// where nothing wider is aligned (W = 1, lead = 2, gap = 1).
template <int DT, int W, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const Args a) {
    pdl_enter();
    const uint64_t i = uint64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= a.work) return;
    const uint32_t rest = fastdiv_u32(uint32_t(i), a.by_units);
    const uint32_t unit = uint32_t(i) - rest * a.by_units.d;
    const uint32_t t = fastdiv_u32(rest, a.by_runs);
    const uint32_t h0 = (rest - t * a.by_runs.d) * a.run;
    const uint32_t h1 = min(h0 + a.run, a.heads);
    const uint16_t* x = a.x + int64_t(t) * a.x_token + int64_t(h0) * a.x_head;
    uint16_t* out = a.out + int64_t(t) * a.out_token + int64_t(h0) * a.out_head;
    if (unit < a.rot_units) {
        constexpr int P = INTERLEAVED ? W / 2 : W;
        const int64_t position = __ldg(a.positions + t);
        float c[P], s[P];
#pragma unroll
        for (int k = 0; k < P; ++k) {
            cos_sin(position, __ldg(a.frequencies + unit * P + k), c[k], s[k]);
            c[k] = __fmul_rn(c[k], a.magnitude);
            s[k] = __fmul_rn(s[k], a.sine_sign * a.magnitude);
        }
        x += unit * (INTERLEAVED ? W : a.lead);
        out += unit * (INTERLEAVED ? W : a.lead);
        for (uint32_t h = h0; h < h1; h += kBatch) {
            const uint32_t n = min(uint32_t(kBatch), h1 - h);
            Piece<W> u[kBatch], v[INTERLEAVED ? 1 : kBatch];
#pragma unroll
            for (uint32_t b = 0; b < kBatch; ++b)
                if (b < n) {
                    u[b] = load<W>(x + b * a.x_head);
                    if constexpr (!INTERLEAVED) v[b] = load<W>(x + b * a.x_head + a.gap);
                }
#pragma unroll
            for (uint32_t b = 0; b < kBatch; ++b)
                if (b < n) {
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        if constexpr (INTERLEAVED) turn<DT>(u[b].v[2 * k], u[b].v[2 * k + 1], c[k], s[k]);
                        else turn<DT>(u[b].v[k], v[b].v[k], c[k], s[k]);
                    }
                    store<W>(out + b * a.out_head, u[b]);
                    if constexpr (!INTERLEAVED) store<W>(out + b * a.out_head + a.gap, v[b]);
                }
            x += kBatch * a.x_head;
            out += kBatch * a.out_head;
        }
    } else {
        const uint32_t at = a.rotated + (unit - a.rot_units) * W;
        for (uint32_t h = h0; h < h1; h += kBatch) {
            const uint32_t n = min(uint32_t(kBatch), h1 - h);
            Piece<W> u[kBatch];
#pragma unroll
            for (uint32_t b = 0; b < kBatch; ++b)
                if (b < n) u[b] = load<W>(x + b * a.x_head + at);
#pragma unroll
            for (uint32_t b = 0; b < kBatch; ++b)
                if (b < n) store<W>(out + b * a.out_head + at, u[b]);
            x += kBatch * a.x_head;
            out += kBatch * a.out_head;
        }
    }
}

}  // namespace rotary
}  // namespace mhc
