// Launch shapes of the cross entropy over a vocabulary.
#include "mhc_entropy.cuh"
#include "mhc_linear_launch.cuh"

namespace mhc {
namespace layer {

namespace {

template <int END, int OUT, int LAYOUT>
cudaError_t launch_end(bool pair, const TileArgs& a, const CUtensorMap& mp, const CUtensorMap& mq, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed[2];
    if (!pair) return launch_split_kernel(split_kernel<false, OUT, LAYOUT, END>, allowed[0], a, mp, mq, stream);
    return launch_pair_kernel(pair_kernel<false, OUT, LAYOUT, false, END>, allowed[1], a, pairs_of(a), mp, mq, stream);
}

// A product of 16-bit operands that ends in `end`.
template <int END, int LAYOUT>
cudaError_t product_into(const Product& p, const EndArgs& end, int dtype, cudaStream_t stream) {
    TileArgs a;
    CUtensorMap mp, mq;
    const Plan plan = plan_of(p.N, p.M, k_blocks(p, dtype), p.a_mn, false);
    const cudaError_t e = lay_out(p, dtype, plan, a, mp, mq);
    if (e != cudaSuccess) return e;
    a.end = end;
    return dtype == kBF16 ? launch_end<END, kBF16, LAYOUT>(plan.pair, a, mp, mq, stream)
                          : launch_end<END, kF16, LAYOUT>(plan.pair, a, mp, mq, stream);
}

// Entries of the vocabulary of a tile.  The groups that are summed together
// are a quarter of it, so it follows from V alone (a token's loss has the same
// bits in every batch): 256 where that gives every pair of CTAs a tile
// whatever the number of tokens, 128 below.
uint32_t entropy_width(int64_t V) { return V >= 256 * kPairsAtOnce ? 256 : 128; }

}  // namespace

int64_t entropy_groups(int64_t V) {
    const int64_t group = entropy_width(V) / 4;
    return (V + group - 1) / group;
}

cudaError_t entropy_fwd(const EntropyCall& c, float* loss, float* lse, float2* partial, float* at) {
    Product p;
    p.a = c.w, p.a_stride = c.w_stride, p.a_mn = false;
    p.b = c.x, p.b_stride = c.x_stride, p.b_mn = false;
    p.M = c.V, p.N = c.T, p.K = c.I, p.by_row = true;
    p.e = {};
    TileArgs a;
    CUtensorMap mp, mq;
    const uint32_t runs = uint32_t((k_blocks(p, c.dtype) + kEntropyRun - 1) / kEntropyRun);
    cudaError_t e = lay_out(p, c.dtype, {true, entropy_width(c.V), runs}, a, mp, mq);
    if (e != cudaSuccess) return e;
    a.end = {};
    a.end.partial = partial, a.end.at = at, a.end.target = c.target;
    static std::atomic<uint64_t> allowed{0};
    e = launch_pair_kernel(pair_kernel<false, kBF16, kBothK, false, kEndEntropy>, allowed, a, pairs_of(a), mp, mq, c.stream);
    if (e != cudaSuccess) return e;
    return launch(entropy::join_kernel, uint32_t((c.T + 31) / 32), 32 * entropy::kWorkers, c.stream, partial, at, c.target,
                  loss, lse, c.T, c.V, uint32_t(entropy_groups(c.V)));
}

cudaError_t entropy_tokens(const EntropyCall& c, const float* grad_loss, const float* grad_lse, const float* lse,
                           EntropyToken* tokens, float* factor) {
    return launch(entropy::token_kernel, 1, entropy::kTokenThreads, c.stream, grad_loss, grad_lse, c.target, lse, tokens,
                  factor, c.T, c.V);
}

cudaError_t entropy_logit_grad(const EntropyCall& c, const EntropyToken* tokens, int64_t first, int64_t count, uint16_t* d,
                               int64_t pitch) {
    Product p;
    p.a = c.x, p.a_stride = c.x_stride, p.a_mn = false;
    p.b = static_cast<const uint16_t*>(c.w) + first * c.w_stride, p.b_stride = c.w_stride, p.b_mn = false;
    p.M = c.T, p.N = count, p.K = c.I, p.by_row = false;
    p.e = {};
    p.e.y = d;
    EndArgs end = {};
    end.tokens = tokens, end.first = int32_t(first), end.pitch = pitch;
    return product_into<kEndProb, kBothK>(p, end, c.dtype, c.stream);
}

cudaError_t entropy_grad_x(const EntropyCall& c, const uint16_t* d, int64_t pitch, int64_t first, int64_t count,
                           const float* sum_in, float* sum_out, const float* factor, void* grad_x) {
    Product p;   // [T,I] += d [T,count] . w[first ..] [count,I]
    p.a = d, p.a_stride = pitch, p.a_mn = false;
    p.b = static_cast<const uint16_t*>(c.w) + first * c.w_stride, p.b_stride = c.w_stride, p.b_mn = true;
    p.M = c.T, p.N = c.I, p.K = count, p.by_row = false;
    p.e = {};
    p.e.y = static_cast<uint16_t*>(grad_x);
    EndArgs end = {};
    end.sum_in = sum_in, end.sum_out = sum_out, end.factor = factor;
    return product_into<kEndSum, kPMnQK>(p, end, c.dtype, c.stream);
}

cudaError_t entropy_grad_w(const EntropyCall& c, const uint16_t* d, int64_t pitch, int64_t first, int64_t count,
                           const float* factor, void* grad_w) {
    Product p;   // [count,I] = d^T [count,T] . x [T,I]
    p.a = d, p.a_stride = pitch, p.a_mn = true;
    p.b = c.x, p.b_stride = c.x_stride, p.b_mn = true;
    p.M = count, p.N = c.I, p.K = c.T, p.by_row = false;
    p.e = {};
    p.e.y = static_cast<uint16_t*>(grad_w) + first * c.I;
    EndArgs end = {};
    end.factor = factor;
    return product_into<kEndSum, kBothMn>(p, end, c.dtype, c.stream);
}

}  // namespace layer
}  // namespace mhc
