// Launch shapes of the matrix product.
#include "mhc_layer_launch.cuh"

namespace mhc {
namespace layer {

using namespace linear;

cudaError_t product(const Product& p, int in, int out, cudaStream_t stream) {
    const dim3 grid(uint32_t((p.N + 63) / 64), uint32_t((p.M + 63) / 64));
    if (in == kE4m3)
        return out == kBF16 ? launch2d(simple_kernel<kE4m3, kBF16>, grid, 256, stream, p)
                            : launch2d(simple_kernel<kE4m3, kF16>, grid, 256, stream, p);
    return in == kBF16 ? launch2d(simple_kernel<kBF16, kBF16>, grid, 256, stream, p)
                       : launch2d(simple_kernel<kF16, kF16>, grid, 256, stream, p);
}

// Runs of rows whose column sums are added up one after the other: 64 rows
// or more each, at most 64 runs (a constant, so that the order of the sum
// depends on T alone).
int64_t slope_partials(int64_t T) {
    const int64_t n = (T + 63) / 64;
    return n < 1 ? 1 : n > 64 ? 64 : n;
}

cudaError_t slope(const uint16_t* g, const uint16_t* preact, uint16_t* u, float* grad_bias, float* partial, int64_t T,
                  int64_t O, int act, int dtype, cudaStream_t stream) {
    const int64_t runs = slope_partials(T), rows = (T + runs - 1) / runs;
    float* sums = grad_bias == nullptr ? nullptr : runs > 1 ? partial : grad_bias;
    const bool vec = O % 8 == 0 && aligned(g, 16) && aligned(preact, 16) && aligned(u, 16);   // null is aligned
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(uint32_t((O + (vec ? 255 : 31)) / (vec ? 256 : 32)), uint32_t(runs));
    cfg.blockDim = dim3(32, kSlopeRows);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto* kernel = dtype == kBF16 ? (vec ? slope_kernel<kBF16, 8> : slope_kernel<kBF16, 1>)
                                  : (vec ? slope_kernel<kF16, 8> : slope_kernel<kF16, 1>);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, g, preact, u, sums, T, O, rows, act);
    if (e != cudaSuccess || grad_bias == nullptr || runs == 1) return e;
    return column_sum(partial, grad_bias, uint32_t(runs), O, stream);
}

}  // namespace layer
}  // namespace mhc
