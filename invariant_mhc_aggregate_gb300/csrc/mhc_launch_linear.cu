// Launch shapes of the matrix product.
#include "mhc_linear_launch.cuh"

namespace mhc {
namespace layer {

namespace {

// Set to 1 when a bounded wait runs out (see mhc_bulk.cuh); one per device.
__device__ unsigned int g_timeouts;

}  // namespace

cudaError_t timeouts_ptr(unsigned int** p) {
    static std::atomic<unsigned int*> cached[kMaxDevices];
    const int dev = current_device();
    if (dev < 0) return cudaErrorInvalidDevice;
    unsigned int* q = cached[dev].load(std::memory_order_acquire);
    if (q == nullptr) {
        const cudaError_t e = cudaGetSymbolAddress(reinterpret_cast<void**>(&q), g_timeouts);
        if (e != cudaSuccess) return e;
        cached[dev].store(q, std::memory_order_release);
    }
    *p = q;
    return cudaSuccess;
}

namespace {

template <bool FP8, int OUT, int LAYOUT>
cudaError_t launch_split(const TileArgs& a, CUtensorMap& mp, CUtensorMap& mq, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed{0};
    return launch_split_kernel(split_kernel<FP8, OUT, LAYOUT>, allowed, a, mp, mq, stream);
}

template <bool FP8, int OUT, int LAYOUT>
cudaError_t launch_pair(const TileArgs& a, CUtensorMap& mp, CUtensorMap& mq, cudaStream_t stream) {
    const uint32_t tiles = a.p_tiles * a.q_tiles, pairs = uint32_t(num_sms()) / 2;
    const uint32_t most = tiles < pairs ? tiles : pairs;
    if (a.splits > 1) {
        static std::atomic<uint64_t> allowed{0};
        return launch_pair_kernel(pair_kernel<FP8, OUT, LAYOUT, true>, allowed, a, most, mp, mq, stream);
    }
    static std::atomic<uint64_t> allowed{0};
    return launch_pair_kernel(pair_kernel<FP8, OUT, LAYOUT, false>, allowed, a, most, mp, mq, stream);
}

template <bool FP8, int OUT, int LAYOUT>
cudaError_t launch_tile(bool pair, const TileArgs& a, CUtensorMap& mp, CUtensorMap& mq, cudaStream_t stream) {
    return pair ? launch_pair<FP8, OUT, LAYOUT>(a, mp, mq, stream) : launch_split<FP8, OUT, LAYOUT>(a, mp, mq, stream);
}

template <int OUT>
cudaError_t launch_layout(bool pair, const TileArgs& a, CUtensorMap& mp, CUtensorMap& mq, bool p_mn, bool q_mn,
                          cudaStream_t stream) {
    if (!p_mn) return launch_tile<false, OUT, kBothK>(pair, a, mp, mq, stream);
    return q_mn ? launch_tile<false, OUT, kBothMn>(pair, a, mp, mq, stream)
                : launch_tile<false, OUT, kPMnQK>(pair, a, mp, mq, stream);
}

}  // namespace

int64_t take_wait_timeouts() {
    unsigned int n = 0;
    const unsigned int zero = 0;
    if (cudaDeviceSynchronize() != cudaSuccess) return -1;
    if (cudaMemcpyFromSymbol(&n, g_timeouts, sizeof(n)) != cudaSuccess) return -1;
    if (n != 0 && cudaMemcpyToSymbol(g_timeouts, &zero, sizeof(zero)) != cudaSuccess) return -1;
    return int64_t(n);
}

cudaError_t product(const Product& p, int in, int out, cudaStream_t stream) {
    return product(p, plan_of(p.N, p.M, k_blocks(p, in), p.a_mn, p.by_row), in, out, stream);
}

cudaError_t product(const Product& p, const Plan& plan, int in, int out, cudaStream_t stream) {
    TileArgs a;
    CUtensorMap mp, mq;
    const cudaError_t e = lay_out(p, in, plan, a, mp, mq);
    if (e != cudaSuccess) return e;
    a.end = {};
    if (in == kE4m3)
        return out == kBF16 ? launch_tile<true, kBF16, kBothK>(plan.pair, a, mp, mq, stream)
                            : launch_tile<true, kF16, kBothK>(plan.pair, a, mp, mq, stream);
    return out == kBF16 ? launch_layout<kBF16>(plan.pair, a, mp, mq, p.b_mn, p.a_mn, stream)
                        : launch_layout<kF16>(plan.pair, a, mp, mq, p.b_mn, p.a_mn, stream);
}

cudaError_t repack(const RepackCall* calls, int count, cudaStream_t stream) {
    Repack r[2] = {};
    uint64_t blocks[2] = {0, 0};
    for (int i = 0; i < count; ++i) {
        const RepackCall& c = calls[i];
        r[i].src = static_cast<const char*>(c.src);
        r[i].dst = static_cast<char*>(c.dst);
        r[i].per_row = uint32_t(c.pitch / 16);
        r[i].vectors = uint64_t(c.rows) * r[i].per_row;
        r[i].by_row = make_fastdiv_u32(r[i].per_row);
        r[i].length = uint64_t(c.length), r[i].stride = uint64_t(c.stride);
        r[i].bytes = uint64_t(c.rows - 1) * r[i].stride + r[i].length;
        blocks[i] = (r[i].vectors + kRepackThreads * kRepackVectors - 1) / (kRepackThreads * kRepackVectors);
    }
    if (blocks[0] + blocks[1] > 0x7FFFFFFFull) return cudaErrorInvalidValue;
    return launch(repack_kernel, uint32_t(blocks[0] + blocks[1]), kRepackThreads, stream, r[0], r[1], uint32_t(blocks[0]));
}

namespace {

template <int DT, int W>
auto slope_kernel_of(int act) {
    switch (act) {
        case kActRelu: return slope_kernel<DT, W, kActRelu>;
        case kActSilu: return slope_kernel<DT, W, kActSilu>;
        case kActGelu: return slope_kernel<DT, W, kActGelu>;
        default: return slope_kernel<DT, W, kActNone>;
    }
}

}  // namespace

// Runs of rows whose column sums are added up one after the other: 64 rows
// or more each, at most 64 runs (a constant, so that the order of the sum
// depends on T alone).
int64_t slope_partials(int64_t T) {
    const int64_t n = (T + 63) / 64;
    return n < 1 ? 1 : n > 64 ? 64 : n;
}

cudaError_t slope(const uint16_t* g, const uint16_t* preact, uint16_t* u, float* grad_bias, float* partial, int64_t T,
                  int64_t O, int64_t pitch, int act, int dtype, cudaStream_t stream) {
    const int64_t runs = slope_partials(T), rows = (T + runs - 1) / runs;
    float* sums = grad_bias == nullptr ? nullptr : runs > 1 ? partial : grad_bias;
    const bool vec = O % 8 == 0 && pitch % 8 == 0 && aligned(g, 16) && aligned(preact, 16) && aligned(u, 16);   // null is aligned
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(uint32_t((O + (vec ? 255 : 31)) / (vec ? 256 : 32)), uint32_t(runs));
    cfg.blockDim = dim3(32, kSlopeRows);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto* kernel = dtype == kBF16 ? (vec ? slope_kernel_of<kBF16, 8>(act) : slope_kernel_of<kBF16, 1>(act))
                                  : (vec ? slope_kernel_of<kF16, 8>(act) : slope_kernel_of<kF16, 1>(act));
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, g, preact, u, sums, T, O, pitch, rows);
    if (e != cudaSuccess || grad_bias == nullptr || runs == 1) return e;
    return column_sum(partial, grad_bias, uint32_t(runs), O, O, stream);
}

}  // namespace layer
}  // namespace mhc
