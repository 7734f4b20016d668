// Launch shapes of the RMS norm kernels.
#include "mhc_layer_launch.cuh"

namespace mhc {
namespace layer {

using namespace norm;

namespace {

// Threads of a row and chunks of a thread: they fix the order of the row's
// sum, so they follow from H alone.  Up to 1024 values a warp holds the row;
// longer rows take 2 chunks a thread, past 8192 values 4, past 16384 values 8.
struct Shape {
    uint32_t nt;
    int K;
};

Shape shape_of(uint32_t H) {
    const uint32_t chunks = (H + 7) / 8;
    if (chunks <= 32) return {32, 1};
    if (chunks <= 64) return {32, 2};
    if (chunks <= 128) return {32, 4};
    if (chunks <= 1024) return {(chunks + 63) / 64 * 32, 2};
    if (chunks <= 2048) return {(chunks + 127) / 128 * 32, 4};
    return {kMaxThreads, 8};
}

constexpr uint32_t kWarpRows = 4;   // rows of a block where a warp holds a row

// Shared memory of one SM that the blocks of these kernels share out.
constexpr uint32_t kRowSmem = 216 * 1024;

template <typename... Params, typename... Args>
cudaError_t launch_rows(void (*kernel)(Params...), uint32_t grid, uint32_t nt, uint32_t rows, uint32_t smem,
                        std::atomic<uint64_t>& allowed, cudaStream_t stream, Args... args) {
    if (smem > 48 * 1024) {
        const cudaError_t e = allow_smem(kernel, kRowSmem, allowed);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(nt, rows);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// The ring kernels' shape: blocks of an SM and stages of a block, so that the
// ring of each SM holds most of its shared memory.
struct RingShape {
    uint32_t blocks, stages;   // blocks: of one SM
};

// `most`: blocks of an SM that the kernel's registers allow.
RingShape ring_shape(uint32_t row_bytes, uint32_t most) {
    const uint32_t fit = kRowSmem / (2 * row_bytes + 1024);   // with two stages each
    RingShape r;
    r.blocks = fit < 1 ? 1 : fit < most ? fit : most;
    r.stages = kRowSmem / r.blocks / row_bytes;
    if (r.stages > kRingStages) r.stages = kRingStages;
    return r;
}

template <int DT, int K, bool VEC, int OUT>
cudaError_t fwd_launch(const FwdArgs& args, Shape s, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed{0};
    const uint32_t rows = s.nt == 32 ? kWarpRows : 1;
    const int64_t most = int64_t(0x7FFFFFFF) * rows;   // rows of one launch
    for (int64_t t0 = 0; t0 < args.T; t0 += most) {
        FwdArgs a = args;
        a.T = args.T - t0 < most ? args.T - t0 : most;
        a.x += t0 * a.x_stride;
        if (a.residual != nullptr) {
            a.residual += t0 * a.residual_stride;
            a.total += t0 * int64_t(a.H);
        }
        a.y = static_cast<char*>(a.y) + t0 * int64_t(a.H) * (OUT == kOutSame ? 2 : 1);
        a.rstd += t0;
        if (OUT != kOutSame) a.scale += t0 * (OUT == kOutFp8Row ? 1 : (int64_t(a.H) + kGroup - 1) / kGroup);
        const cudaError_t e = launch_rows(fwd_kernel<DT, K, VEC, OUT>, uint32_t((a.T + rows - 1) / rows), s.nt, rows, 0,
                                          allowed, stream, a);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <int DT, int K, int OUT>
cudaError_t fwd_ring(FwdArgs a, Shape s, RingShape ring, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed{0}, narrow{0};
    const cudaError_t e = timeouts_ptr(&a.timeouts);
    if (e != cudaSuccess) return e;
    RingRows r = {{a.x, a.residual, nullptr}, {a.x_stride, a.residual_stride, 0}, a.residual != nullptr ? 2u : 1u};
    // four times the blocks that run at once: as they end one by one, the next
    // ones start under the others' rows, and the last rows spread out (T = 4096,
    // H = 7168: 44.3 us with one round of blocks, 40.6 with two, 38.7 with four)
    const int64_t most = int64_t(num_sms()) * ring.blocks * 4;
    const uint32_t grid = uint32_t(a.T < most ? a.T : most), smem = ring.stages * r.arrays * a.H * 2;
    if (K == 2 && s.nt <= 448)
        return launch_rows(fwd_ring_kernel<DT, K, OUT, 448>, grid, s.nt, 1, smem, narrow, stream, a, r, ring.stages);
    return launch_rows(fwd_ring_kernel<DT, K, OUT, 512>, grid, s.nt, 1, smem, allowed, stream, a, r, ring.stages);
}

template <int DT, int K, bool VEC>
cudaError_t fwd_out(const FwdArgs& a, Shape s, int out, cudaStream_t stream) {
    if constexpr (VEC && (K == 2 || K == 4)) {
        const uint32_t row = a.H * 2 * (a.residual != nullptr ? 2 : 1);
        const RingShape ring = ring_shape(row, K == 2 ? 65536 / (s.nt * (s.nt <= 448 ? 72 : 64)) : 1);
        // (not for rows of one warp, nor where a block would have no second row)
        if (s.nt > 32 && ring.stages >= 2 && a.T > int64_t(num_sms()) * ring.blocks) switch (out) {
            case kOutSame: return fwd_ring<DT, K, kOutSame>(a, s, ring, stream);
            case kOutFp8Row: return fwd_ring<DT, K, kOutFp8Row>(a, s, ring, stream);
            default: return fwd_ring<DT, K, kOutFp8Group>(a, s, ring, stream);
        }
    }
    switch (out) {
        case kOutSame: return fwd_launch<DT, K, VEC, kOutSame>(a, s, stream);
        case kOutFp8Row: return fwd_launch<DT, K, VEC, kOutFp8Row>(a, s, stream);
        default: return fwd_launch<DT, K, VEC, kOutFp8Group>(a, s, stream);
    }
}

template <int DT, bool VEC>
cudaError_t fwd_shape(const FwdArgs& a, int out, cudaStream_t stream) {
    const Shape s = shape_of(a.H);
    switch (s.K) {
        case 1: return fwd_out<DT, 1, VEC>(a, s, out, stream);
        case 2: return fwd_out<DT, 2, VEC>(a, s, out, stream);
        case 4: return fwd_out<DT, 4, VEC>(a, s, out, stream);
        default: return fwd_out<DT, 8, VEC>(a, s, out, stream);
    }
}

template <int DT, int K, bool VEC>
cudaError_t bwd_launch(BwdArgs a, Shape s, uint32_t blocks, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed{0};
    const uint32_t rows = s.nt == 32 ? kWarpRows : 1;
    if constexpr (VEC && (K == 2 || K == 4)) {
        const RingRows r = {{a.g, a.s, a.grad_total}, {a.g_stride, a.s_stride, int64_t(a.H)}, a.grad_total != nullptr ? 3u : 2u};
        const uint32_t row = a.H * 2 * r.arrays;
        constexpr uint32_t kStages = 2;   // a third: 48.3 us against 46.0 at T = 4096, H = 7168
        if (rows == 1 && kStages * row <= kRowSmem && a.T > int64_t(blocks)) {
            static std::atomic<uint64_t> ring_allowed{0};
            const cudaError_t e = timeouts_ptr(&a.timeouts);
            if (e != cudaSuccess) return e;
            return launch_rows(bwd_ring_kernel<DT, K>, blocks, s.nt, 1, kStages * row, ring_allowed, stream, a, r, kStages);
        }
    }
    return launch_rows(bwd_kernel<DT, K, VEC>, blocks, s.nt, rows, rows == 1 ? 0 : 8u * K * 32 * 4, allowed,
                       stream, a);
}

template <int DT, bool VEC>
cudaError_t bwd_shape(const BwdArgs& a, uint32_t blocks, cudaStream_t stream) {
    const Shape s = shape_of(a.H);
    switch (s.K) {
        case 1: return bwd_launch<DT, 1, VEC>(a, s, blocks, stream);
        case 2: return bwd_launch<DT, 2, VEC>(a, s, blocks, stream);
        case 4: return bwd_launch<DT, 4, VEC>(a, s, blocks, stream);
        default: return bwd_launch<DT, 8, VEC>(a, s, blocks, stream);
    }
}

bool rows16(const void* p, int64_t stride) { return aligned(p, 16) && stride % 8 == 0; }

}  // namespace

cudaError_t norm_fwd(const FwdArgs& a, int dtype, int out, cudaStream_t stream) {
    const bool vec = a.H % 8 == 0 && rows16(a.x, a.x_stride) && aligned(a.weight, 16) && aligned(a.y, 16) &&
                     (a.residual == nullptr || (rows16(a.residual, a.residual_stride) && aligned(a.total, 16)));
    if (dtype == kBF16) return vec ? fwd_shape<kBF16, true>(a, out, stream) : fwd_shape<kBF16, false>(a, out, stream);
    return vec ? fwd_shape<kF16, true>(a, out, stream) : fwd_shape<kF16, false>(a, out, stream);
}

// Blocks of the backward, each with a partial sum of grad_weight: for each of
// 152 SMs as many as its registers run at once, 512 threads' worth and at most
// four (a constant, so that the sum's order does not depend on the device), and
// no more than have rows.  T = 4096, H = 7168: 46.0 us with one an SM, 48.2 with
// two, 53.7 with four; T = 16384, H = 2048: 51.3 with four, 67.8 with two.
uint32_t norm_bwd_partials(int64_t T, int64_t H) {
    const Shape s = shape_of(uint32_t(H));
    const uint32_t rows = s.nt == 32 ? kWarpRows : 1, fit = 512 / (s.nt * rows);
    const int64_t most = 152 * (fit < 1 ? 1 : fit > 4 ? 4 : fit);
    const int64_t blocks = (T + rows - 1) / rows;
    return uint32_t(blocks < most ? blocks : most);
}

cudaError_t norm_bwd(BwdArgs a, float* grad_weight, float* workspace, int dtype, cudaStream_t stream) {
    const uint32_t P = norm_bwd_partials(a.T, a.H);
    a.partial = P > 1 ? workspace : grad_weight;
    a.pitch = (a.H + 7) / 8 * 8;   // whole chunks
    const bool vec = a.H % 8 == 0 && rows16(a.g, a.g_stride) && rows16(a.s, a.s_stride) && aligned(a.weight, 16) &&
                     aligned(a.grad_x, 16) && aligned(a.partial, 16) &&
                     (a.grad_total == nullptr || aligned(a.grad_total, 16));
    cudaError_t e;
    if (dtype == kBF16) e = vec ? bwd_shape<kBF16, true>(a, P, stream) : bwd_shape<kBF16, false>(a, P, stream);
    else e = vec ? bwd_shape<kF16, true>(a, P, stream) : bwd_shape<kF16, false>(a, P, stream);
    if (e != cudaSuccess || P <= 1) return e;
    return column_sum(workspace, grad_weight, P, a.H, a.pitch, stream);
}

cudaError_t column_sum(const float* partial, float* out, uint32_t P, int64_t H, int64_t pitch, cudaStream_t stream) {
    const uint32_t blocks = uint32_t((H + 31) / 32);
    return pitch % 4 == 0 && aligned(partial, 16)
               ? launch(column_sum_kernel<true>, blocks, 8 * kColGroups, stream, partial, out, P, uint32_t(H), uint32_t(pitch))
               : launch(column_sum_kernel<false>, blocks, 8 * kColGroups, stream, partial, out, P, uint32_t(H),
                        uint32_t(pitch));
}

}  // namespace layer
}  // namespace mhc
