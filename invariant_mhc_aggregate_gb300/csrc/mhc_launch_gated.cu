// Launch shapes of the gated product.
#include "mhc_gated.cuh"
#include "mhc_linear_launch.cuh"

namespace mhc {
namespace layer {

namespace {

template <bool FP8, int OUT>
cudaError_t launch_gated(bool pair, const TileArgs& a, const CUtensorMap& mp, const CUtensorMap& mq, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed[3];
    if (!pair) return launch_split_kernel(split_kernel<FP8, OUT, kBothK, kEndGated>, allowed[0], a, mp, mq, stream, kGatedBytes);
    if (a.splits > 1)
        return launch_pair_kernel(pair_kernel<FP8, OUT, kBothK, true, kEndGated>, allowed[1], a, pairs_of(a), mp, mq, stream,
                                  kGatedBytes);
    return launch_pair_kernel(pair_kernel<FP8, OUT, kBothK, false, kEndGated>, allowed[2], a, pairs_of(a), mp, mq, stream,
                              kGatedBytes);
}

template <int DT, int W>
auto slope_kernel_of(int act) {
    switch (act) {
        case kActRelu: return gated::slope_kernel<DT, W, kActRelu>;
        case kActSilu: return gated::slope_kernel<DT, W, kActSilu>;
        case kActGelu: return gated::slope_kernel<DT, W, kActGelu>;
        default: return gated::slope_kernel<DT, W, kActNone>;
    }
}

}  // namespace

cudaError_t gated_product(const Product& p, int in, int out, cudaStream_t stream) {
    TileArgs a;
    CUtensorMap mp, mq;
    const Plan plan = plan_of(p.N, p.M, k_blocks(p, in), false, true);
    const bool few = p.M <= kFewRows && plan.splits == 1;   // (parts of K are faster in a cluster's CTAs)
    cudaError_t e = few ? lay_out_few(p, in, few_lanes(p.N), plan.splits, a, mp, mq) : lay_out(p, in, plan, a, mp, mq);
    if (e != cudaSuccess) return e;
    // half a tile's lanes a copy: rows of the gate (past its end, of the up projection: nobody's lanes), then of the up
    // projection (past its end, zeros)
    e = encode(&mp, p.b, p.N, p.K, p.b_stride, in == kE4m3 ? 1 : 2, a.lanes / 2);
    if (e != cudaSuccess) return e;
    a.p_box = kLanesP;   // (two boxes)
    a.end = {};
    a.end.half = p.N / 2;
    if (few) {
        if (in == kE4m3)
            return out == kBF16 ? launch_few<true, kBF16, kEndGated>(a, mp, mq, stream)
                                : launch_few<true, kF16, kEndGated>(a, mp, mq, stream);
        return out == kBF16 ? launch_few<false, kBF16, kEndGated>(a, mp, mq, stream)
                            : launch_few<false, kF16, kEndGated>(a, mp, mq, stream);
    }
    if (in == kE4m3)
        return out == kBF16 ? launch_gated<true, kBF16>(plan.pair, a, mp, mq, stream)
                            : launch_gated<true, kF16>(plan.pair, a, mp, mq, stream);
    return out == kBF16 ? launch_gated<false, kBF16>(plan.pair, a, mp, mq, stream)
                        : launch_gated<false, kF16>(plan.pair, a, mp, mq, stream);
}

cudaError_t gated_slope(const uint16_t* g, const uint16_t* preact, uint16_t* u, float* grad_bias, float* partial, int64_t T,
                        int64_t F, int64_t pitch, int act, int dtype, cudaStream_t stream) {
    const int64_t runs = slope_partials(T), rows = (T + runs - 1) / runs;
    float* sums = grad_bias == nullptr ? nullptr : runs > 1 ? partial : grad_bias;
    const bool vec = F % 8 == 0 && pitch % 8 == 0 && aligned(g, 16) && aligned(preact, 16) && aligned(u, 16);   // null is aligned
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(uint32_t((F + (vec ? 255 : 31)) / (vec ? 256 : 32)), uint32_t(runs));
    cfg.blockDim = dim3(32, kSlopeRows);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto* kernel = dtype == kBF16 ? (vec ? slope_kernel_of<kBF16, 8>(act) : slope_kernel_of<kBF16, 1>(act))
                                  : (vec ? slope_kernel_of<kF16, 8>(act) : slope_kernel_of<kF16, 1>(act));
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, g, preact, u, sums, T, F, pitch, rows);
    if (e != cudaSuccess || grad_bias == nullptr || runs == 1) return e;
    return column_sum(partial, grad_bias, uint32_t(runs), 2 * F, 2 * F, stream);
}

}  // namespace layer
}  // namespace mhc
