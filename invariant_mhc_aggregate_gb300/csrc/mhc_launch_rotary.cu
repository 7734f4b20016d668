// Launch shapes of the rotary kernel.
#include "mhc_layer_launch.cuh"
#include "mhc_rotary.cuh"

namespace mhc {
namespace layer {

namespace {

template <int DT, int W>
cudaError_t launch_width(const RotaryCall& c) {
    const bool one_piece = c.interleaved && W > 1;
    const uint32_t rot_units = uint32_t(one_piece ? c.R / W : c.R / (2 * W));
    const uint32_t copied = uint32_t((c.D - c.R) / W), copy_units = one_piece ? copied : (copied + 1) / 2;
    const uint32_t units = rot_units + copy_units;
    // Heads of one thread: 8 share a thread's cosines and sines (their cost
    // is then below that of the values' own arithmetic); fewer where the call
    // would not give each SM 1024 threads.
    const uint64_t want = uint64_t(num_sms()) * 1024;
    uint64_t run = 8;
    while (run > 1 && uint64_t(c.T) * units * ((uint64_t(c.heads) + run - 1) / run) < want) run /= 2;
    const uint64_t runs = (uint64_t(c.heads) + run - 1) / run;
    const uint64_t per_token = runs * units;
    if (per_token > 0x7FFFFFFFull) return cudaErrorInvalidValue;
    const int64_t tokens = int64_t(0x7FFFFFFFull / per_token);   // of one launch: thread indices are 32-bit
    for (int64_t t0 = 0; t0 < c.T; t0 += tokens) {
        const int64_t nt = c.T - t0 < tokens ? c.T - t0 : tokens;
        rotary::Args a;
        a.x = c.x + t0 * c.x_token;
        a.out = c.out + t0 * c.out_token;
        a.positions = c.positions + t0;
        a.frequencies = c.frequencies;
        a.x_token = c.x_token, a.x_head = c.x_head, a.out_token = c.out_token, a.out_head = c.out_head;
        a.work = uint64_t(nt) * per_token;
        a.heads = uint32_t(c.heads), a.D = uint32_t(c.D), a.R = uint32_t(c.R);
        a.copy_gap = copy_units * W;
        a.lead = c.interleaved ? 2 : W;
        a.gap = c.interleaved ? 1 : uint32_t(c.R / 2);
        a.run = uint32_t(run);
        a.rot_units = rot_units;
        a.by_units = make_fastdiv_u32(units);
        a.by_runs = make_fastdiv_u32(uint32_t(runs));
        a.magnitude = c.magnitude;
        a.sine_sign = c.inverse ? -1.0f : 1.0f;
        const uint32_t blocks = uint32_t((a.work + rotary::kThreads - 1) / rotary::kThreads);
        cudaError_t e;
        if constexpr (W > 1)
            e = one_piece ? launch(rotary::rotary_kernel<DT, W, true>, blocks, rotary::kThreads, c.stream, a)
                          : launch(rotary::rotary_kernel<DT, W, false>, blocks, rotary::kThreads, c.stream, a);
        else
            e = launch(rotary::rotary_kernel<DT, 1, false>, blocks, rotary::kThreads, c.stream, a);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Whether every piece of W values starts on a 2 W byte boundary.
bool fits(const RotaryCall& c, int64_t W) {
    return aligned(c.x, 2 * W) && aligned(c.out, 2 * W) && c.x_token % W == 0 && c.x_head % W == 0 &&
           c.out_token % W == 0 && c.out_head % W == 0 && c.D % W == 0 &&
           (c.interleaved ? c.R : c.R / 2) % W == 0;
}

template <int DT>
cudaError_t launch_type(const RotaryCall& c) {
    if (fits(c, 8)) return launch_width<DT, 8>(c);
    if (fits(c, 4)) return launch_width<DT, 4>(c);
    if (fits(c, 2)) return launch_width<DT, 2>(c);
    return launch_width<DT, 1>(c);
}

}  // namespace

cudaError_t rotary(const RotaryCall& c) { return c.dtype == kBF16 ? launch_type<kBF16>(c) : launch_type<kF16>(c); }

}  // namespace layer
}  // namespace mhc
