// What the launches of the product's kernels share (mhc_linear.cuh): tensor
// maps, shared memory, the launch itself.
#pragma once

#include <cudaTypedefs.h>

#include "mhc_few.cuh"
#include "mhc_layer_launch.cuh"
#include "mhc_linear_plan.h"

namespace mhc {
namespace layer {

using namespace linear;

// cuTensorMapEncodeTiled through the runtime's driver entry point (the
// library does not link the driver library itself); resolved once.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
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
inline cudaError_t encode(CUtensorMap* map, const void* base, int64_t rows, int64_t length, int64_t stride, int64_t size,
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
// `beside`: bytes that a kernel wants beside the ring.
inline void set_ring(TileArgs& a, uint32_t block_bytes, uint32_t beside) {
    const uint32_t ring = kRingBytes - beside;
    a.block_bytes = block_bytes;
    a.unit = ring / (2 * block_bytes) >= 3 ? 2 : 1;
    a.stage_bytes = a.unit * block_bytes;
    a.stages = ring / a.stage_bytes < kMaxStages ? ring / a.stage_bytes : kMaxStages;
}

// Shared memory in which the warps of a gated tile exchange its halves.
constexpr uint32_t kGatedBytes = kEpilogueWarps / 4 * kExchange;

// A product's tiles and operands as `plan` lays them out: the arguments and the two tensor maps.
inline cudaError_t lay_out(const Product& p, int in, const Plan& plan, TileArgs& a, CUtensorMap& mp, CUtensorMap& mq) {
    const int64_t size = in == kE4m3 ? 1 : 2;
    const bool p_mn = p.b_mn, q_mn = p.a_mn;
    const uint32_t lanes = plan.pair ? 2 * kLanesP : kLanesP, box_q = plan.pair ? plan.width / 2 : plan.width;
    a.e = p.e;
    a.N = p.N;
    a.rows = uint32_t(p.M);
    a.kb = uint32_t((p.K * size + 127) / 128);
    a.width = plan.width, a.splits = plan.splits, a.lanes = kLanesP;
    a.p_tiles = uint32_t((p.N + lanes - 1) / lanes);
    a.q_tiles = uint32_t((p.M + a.width - 1) / a.width);
    a.idesc = umma::instr_desc(in == kBF16 ? 1 : 0, p_mn, q_mn, lanes, a.width);
    cudaError_t e = timeouts_ptr(&a.timeouts);
    if (e != cudaSuccess) return e;
    a.p_box = plan.pair && !p_mn && p.N < int64_t(kLanesP) ? uint32_t((p.N + 7) / 8 * 8) : kLanesP;
    e = p_mn ? encode(&mp, p.b, p.K, p.N, p.b_stride, size, 64) : encode(&mp, p.b, p.N, p.K, p.b_stride, size, a.p_box);
    if (e != cudaSuccess) return e;
    return q_mn ? encode(&mq, p.a, p.K, p.M, p.a_stride, size, 64) : encode(&mq, p.a, p.M, p.K, p.a_stride, size, box_q);
}

inline int64_t k_blocks(const Product& p, int in) { return (p.K * (in == kE4m3 ? 1 : 2) + 127) / 128; }

// split_kernel and pair_kernel by name: one cluster a tile, or a pair of CTAs for each of `pairs` tiles at a time.
template <typename Kernel>
cudaError_t launch_split_kernel(Kernel kernel, std::atomic<uint64_t>& allowed, TileArgs a, const CUtensorMap& mp, const CUtensorMap& mq,
                                cudaStream_t stream, uint32_t beside = 0) {
    set_ring(a, kBytesP + a.width * 128, beside);
    const uint32_t parts = a.splits > 1 ? a.width * kLanesP * 4 : 0;
    const uint32_t ring = a.stages * a.stage_bytes;
    a.end.exchange = ring > parts ? ring : parts;
    return launch_tiles(kernel, allowed, dim3(a.p_tiles * a.splits, a.q_tiles), kSplitThreads, a.end.exchange + beside + 1024,
                        a.splits, stream, mp, mq, a);
}

template <typename Kernel>
cudaError_t launch_pair_kernel(Kernel kernel, std::atomic<uint64_t>& allowed, TileArgs a, uint32_t pairs, const CUtensorMap& mp,
                               const CUtensorMap& mq, cudaStream_t stream, uint32_t beside = 0) {
    set_ring(a, kBytesP + a.width / 2 * 128, beside);
    a.end.exchange = a.stages * a.stage_bytes;
    return launch_tiles(kernel, allowed, dim3(2 * pairs), kPairThreads, a.end.exchange + beside + 1024, 2, stream, mp, mq, a);
}

// Pairs of CTAs that tiles are given out to.
inline uint32_t pairs_of(const TileArgs& a, uint32_t parts = 1) {
    const uint32_t tiles = a.p_tiles * a.q_tiles * parts, pairs = uint32_t(num_sms()) / 2;
    return tiles < pairs ? tiles : pairs;
}

// few_kernel's tiles and operands: as lay_out, with p.M rows in one tile of
// few_width of them and `lanes` output columns a tile.
inline cudaError_t lay_out_few(const Product& p, int in, uint32_t lanes, uint32_t parts, TileArgs& a, CUtensorMap& mp, CUtensorMap& mq) {
    const int64_t size = in == kE4m3 ? 1 : 2;
    a.e = p.e;
    a.N = p.N;
    a.rows = uint32_t(p.M);
    a.kb = uint32_t((p.K * size + 127) / 128);
    a.width = few_width(p.M), a.lanes = lanes, a.splits = parts;
    a.p_tiles = uint32_t((p.N + lanes - 1) / lanes), a.q_tiles = 1;
    a.idesc = umma::instr_desc(in == kBF16 ? 1 : 0, false, false, kLanesP, a.width);
    cudaError_t e = timeouts_ptr(&a.timeouts);
    if (e != cudaSuccess) return e;
    e = encode(&mp, p.b, p.N, p.K, p.b_stride, size, lanes);
    if (e != cudaSuccess) return e;
    return encode(&mq, p.a, p.M, p.K, p.a_stride, size, a.width);
}

template <bool FP8, int OUT, int WIDTH, int END>
cudaError_t launch_few_width(TileArgs a, const CUtensorMap& mp, const CUtensorMap& mq, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed{0};
    const uint32_t sms = uint32_t(num_sms()), beside = END == kEndGated ? kGatedBytes : 0;
    const uint32_t tiles = END == kEndSum ? a.p_tiles * a.splits : a.p_tiles;
    set_ring(a, kBytesP + WIDTH * 128, beside);
    a.end.exchange = a.stages * a.stage_bytes;
    return launch_tiles(few_kernel<FP8, OUT, WIDTH, END>, allowed, dim3(tiles < sms ? tiles : sms), kFewThreads<WIDTH>,
                        a.end.exchange + beside + 1024, 1, stream, mp, mq, a);
}

template <bool FP8, int OUT, int END>
cudaError_t launch_few(const TileArgs& a, const CUtensorMap& mp, const CUtensorMap& mq, cudaStream_t stream) {
    switch (a.width) {
        case 16: return launch_few_width<FP8, OUT, 16, END>(a, mp, mq, stream);
        case 32: return launch_few_width<FP8, OUT, 32, END>(a, mp, mq, stream);
        default: return launch_few_width<FP8, OUT, 64, END>(a, mp, mq, stream);
    }
}

}  // namespace layer
}  // namespace mhc
