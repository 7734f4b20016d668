// Launch shapes of the RMS norm kernels.
#include "mhc_layer_launch.cuh"

namespace mhc {
namespace layer {

using namespace norm;

namespace {

// Threads of a row and chunks of a thread: they fix the order of the row's
// sum, so they follow from H alone.  Up to 1024 values a warp holds the row;
// longer rows take 4 chunks a thread.
struct Shape {
    uint32_t nt;
    int K;
};

Shape shape_of(uint32_t H) {
    const uint32_t chunks = (H + 7) / 8;
    if (chunks <= 32) return {32, 1};
    if (chunks <= 64) return {32, 2};
    if (chunks <= 128) return {32, 4};
    return {(chunks + 127) / 128 * 32, 4};
}

constexpr uint32_t kWarpRows = 4;   // rows of a block where a warp holds a row

uint32_t stage_bytes(Shape s) { return 8u * uint32_t(s.K) * s.nt * 4u; }

template <typename Args>
cudaError_t launch_rows(void (*kernel)(Args), uint32_t grid, uint32_t nt, uint32_t rows, uint32_t smem,
                        std::atomic<uint64_t>& allowed, cudaStream_t stream, const Args& a) {
    if (smem > 48 * 1024) {
        const cudaError_t e = allow_smem(kernel, 8 * 4 * 1024 * 4, allowed);
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
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int DT, int K, bool VEC, int OUT>
cudaError_t fwd_launch(const FwdArgs& args, Shape s, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed{0};
    const uint32_t rows = VEC && s.nt == 32 ? kWarpRows : 1;
    const uint32_t smem = VEC ? 0 : stage_bytes(s);
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
        const cudaError_t e = launch_rows(fwd_kernel<DT, K, VEC, OUT>, uint32_t((a.T + rows - 1) / rows), s.nt, rows,
                                          smem, allowed, stream, a);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <int DT, int K, bool VEC>
cudaError_t fwd_out(const FwdArgs& a, Shape s, int out, cudaStream_t stream) {
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
        default: return fwd_out<DT, 4, VEC>(a, s, out, stream);
    }
}

template <int DT, int K, bool VEC>
cudaError_t bwd_launch(const BwdArgs& a, Shape s, uint32_t blocks, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed{0};
    const uint32_t rows = VEC && s.nt == 32 ? kWarpRows : 1;
    return launch_rows(bwd_kernel<DT, K, VEC>, blocks, s.nt, rows, VEC && rows == 1 ? 0 : stage_bytes(s), allowed,
                       stream, a);
}

template <int DT, bool VEC>
cudaError_t bwd_shape(const BwdArgs& a, uint32_t blocks, cudaStream_t stream) {
    const Shape s = shape_of(a.H);
    switch (s.K) {
        case 1: return bwd_launch<DT, 1, VEC>(a, s, blocks, stream);
        case 2: return bwd_launch<DT, 2, VEC>(a, s, blocks, stream);
        default: return bwd_launch<DT, 4, VEC>(a, s, blocks, stream);
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

// Blocks of the backward, each with a partial sum of grad_weight: two for
// each of the 152 SMs, a constant so that the sum's order does not depend on
// the device.
uint32_t norm_bwd_partials(int64_t T, int64_t H) {
    (void)H;
    return uint32_t(T < 304 ? T : 304);
}

cudaError_t norm_bwd(BwdArgs a, float* grad_weight, float* workspace, int dtype, cudaStream_t stream) {
    const uint32_t P = norm_bwd_partials(a.T, a.H);
    a.partial = P > 1 ? workspace : grad_weight;
    const bool vec = a.H % 8 == 0 && rows16(a.g, a.g_stride) && rows16(a.s, a.s_stride) && aligned(a.weight, 16) &&
                     aligned(a.grad_x, 16) && aligned(a.partial, 16) &&
                     (a.grad_total == nullptr || aligned(a.grad_total, 16));
    cudaError_t e;
    if (dtype == kBF16) e = vec ? bwd_shape<kBF16, true>(a, P, stream) : bwd_shape<kBF16, false>(a, P, stream);
    else e = vec ? bwd_shape<kF16, true>(a, P, stream) : bwd_shape<kF16, false>(a, P, stream);
    if (e != cudaSuccess || P <= 1) return e;
    return column_sum(workspace, grad_weight, P, a.H, stream);
}

cudaError_t column_sum(const float* partial, float* out, uint32_t P, int64_t H, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(uint32_t((H + 31) / 32));
    cfg.blockDim = dim3(32, kColRows);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, column_sum_kernel, partial, out, P, uint32_t(H));
}

}  // namespace layer
}  // namespace mhc
