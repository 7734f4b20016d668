// Launch shapes of the matrix product.
#include <cudaTypedefs.h>

#include "mhc_layer_launch.cuh"
#include "mhc_linear_plan.h"

namespace mhc {
namespace layer {

using namespace linear;

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

// cuTensorMapEncodeTiled through the runtime's driver entry point (the
// library does not link the driver library itself); resolved once.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static std::atomic<void*> fn{nullptr};
    void* p = fn.load(std::memory_order_acquire);
    if (p == nullptr) {
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(p, std::memory_order_release);
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
}

// Rows of `length` elements of `size` bytes, box 128 bytes x box_rows, 128-byte swizzle.
cudaError_t encode(CUtensorMap* map, const void* base, int64_t rows, int64_t length, int64_t stride, int64_t size,
                   uint32_t box_rows) {
    const PFN_cuTensorMapEncodeTiled_v12000 f = tensor_map_encoder();
    if (f == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {cuuint64_t(length), cuuint64_t(rows)};
    // one row has no stride; any multiple of 16 does
    const cuuint64_t strides[1] = {cuuint64_t((rows > 1 ? stride : (length + 15) / 16 * 16) * size)};
    const cuuint32_t box[2] = {cuuint32_t(128 / size), box_rows};
    const cuuint32_t step[2] = {1, 1};
    // Fetching 256 bytes at a time into L2 pays where every row starts on a sector
    // (T = 4096, 7168 x 7168 225 us, with 128 238) and costs where not (7160 x 7168 285, 274;
    // T = 512, 7160 x 4096 41, 35).
    const bool sectors = strides[0] % 32 == 0 && reinterpret_cast<uintptr_t>(base) % 32 == 0;
    const CUresult r = f(map, size == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2,
                         const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B,
                         sectors ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Shared memory of a ring of stages: 7 stages of the pair kernel's widest
// tile, next to the barriers and the 1024 bytes of alignment in the 227 KB.
constexpr uint32_t kRingBytes = 224 * 1024;

template <typename Kernel>
cudaError_t launch_tiles(Kernel kernel, std::atomic<uint64_t>& allowed, dim3 grid, uint32_t threads, uint32_t smem,
                         uint32_t cluster, cudaStream_t stream, const CUtensorMap& mp, const CUtensorMap& mq,
                         const TileArgs& a) {
    cudaError_t e = allow_smem(kernel, kRingBytes + 1024, allowed);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, mp, mq, a);
}

// The ring's stages.  Two blocks of K a stage halve the waits and signals of
// a block, which take longer than the multiplications of narrow tiles (M = 512
// at 4096 x 4096 32.4 -> 20.8 us, one row at 7168 x 7168 21.7 -> 19.6), where
// three such stages fit: all but split_kernel's widest tiles.
void set_ring(TileArgs& a, uint32_t block_bytes) {
    a.block_bytes = block_bytes;
    a.unit = kRingBytes / (2 * block_bytes) >= 3 ? 2 : 1;
    a.stage_bytes = a.unit * block_bytes;
    a.stages = kRingBytes / a.stage_bytes < kMaxStages ? kRingBytes / a.stage_bytes : kMaxStages;
}

template <bool FP8, int OUT, int LAYOUT>
cudaError_t launch_split(TileArgs a, CUtensorMap& mp, CUtensorMap& mq, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed{0};
    set_ring(a, kBytesP + a.width * 128);
    const uint32_t parts = a.splits > 1 ? a.width * kLanesP * 4 : 0;
    const uint32_t ring = a.stages * a.stage_bytes;
    return launch_tiles(split_kernel<FP8, OUT, LAYOUT>, allowed, dim3(a.p_tiles * a.splits, a.q_tiles), kSplitThreads,
                        (ring > parts ? ring : parts) + 1024, a.splits, stream, mp, mq, a);
}

template <bool FP8, int OUT, int LAYOUT>
cudaError_t launch_pair(TileArgs a, CUtensorMap& mp, CUtensorMap& mq, cudaStream_t stream) {
    set_ring(a, kBytesP + a.width / 2 * 128);
    const uint32_t tiles = a.p_tiles * a.q_tiles, pairs = uint32_t(num_sms()) / 2;
    const dim3 grid(2 * (tiles < pairs ? tiles : pairs));
    const uint32_t smem = a.stages * a.stage_bytes + 1024;
    if (a.splits > 1) {
        static std::atomic<uint64_t> allowed{0};
        return launch_tiles(pair_kernel<FP8, OUT, LAYOUT, true>, allowed, grid, kPairThreads, smem, 2, stream, mp, mq, a);
    }
    static std::atomic<uint64_t> allowed{0};
    return launch_tiles(pair_kernel<FP8, OUT, LAYOUT, false>, allowed, grid, kPairThreads, smem, 2, stream, mp, mq, a);
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
    const bool fp8 = in == kE4m3;
    const int64_t size = fp8 ? 1 : 2;
    TileArgs a;
    a.e = p.e;
    a.N = p.N;
    a.rows = uint32_t(p.M);
    a.kb = uint32_t((p.K * size + 127) / 128);
    const bool p_mn = p.b_mn, q_mn = p.a_mn;
    cudaError_t e = timeouts_ptr(&a.timeouts);
    if (e != cudaSuccess) return e;
    const Plan plan = plan_of(p.N, p.M, a.kb, q_mn, p.by_row);
    const bool pair = plan.pair;
    const uint32_t lanes = pair ? 2 * kLanesP : kLanesP, box_q = pair ? plan.width / 2 : plan.width;
    a.width = plan.width, a.splits = plan.splits;
    a.p_tiles = uint32_t((p.N + lanes - 1) / lanes);
    a.q_tiles = uint32_t((p.M + a.width - 1) / a.width);
    a.idesc = umma::instr_desc(in == kBF16 ? 1 : 0, p_mn, q_mn, lanes, a.width);
    CUtensorMap mp, mq;
    e = p_mn ? encode(&mp, p.b, p.K, p.N, p.b_stride, size, 64) : encode(&mp, p.b, p.N, p.K, p.b_stride, size, kLanesP);
    if (e != cudaSuccess) return e;
    e = q_mn ? encode(&mq, p.a, p.K, p.M, p.a_stride, size, 64) : encode(&mq, p.a, p.M, p.K, p.a_stride, size, box_q);
    if (e != cudaSuccess) return e;
    if (fp8)
        return out == kBF16 ? launch_tile<true, kBF16, kBothK>(pair, a, mp, mq, stream)
                            : launch_tile<true, kF16, kBothK>(pair, a, mp, mq, stream);
    return out == kBF16 ? launch_layout<kBF16>(pair, a, mp, mq, p_mn, q_mn, stream)
                        : launch_layout<kF16>(pair, a, mp, mq, p_mn, q_mn, stream);
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
        blocks[i] = (r[i].vectors + kRepackThreads - 1) / kRepackThreads;
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
