// Launch shapes of the cross entropy over a vocabulary.
#include "mhc_entropy.cuh"
#include "mhc_linear_launch.cuh"

namespace mhc {
namespace layer {

namespace {

template <int END, int LAYOUT, bool PARTS = false>
cudaError_t launch_end(const TileArgs& a, int dtype, uint32_t pairs, const CUtensorMap& mp, const CUtensorMap& mq, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed[2];
    if (dtype == kBF16) return launch_pair_kernel(pair_kernel<false, kBF16, LAYOUT, PARTS, END>, allowed[0], a, pairs, mp, mq, stream);
    return launch_pair_kernel(pair_kernel<false, kF16, LAYOUT, PARTS, END>, allowed[1], a, pairs, mp, mq, stream);
}

// A sum over tokens by itself, in parts one after the other where there are many (kSumBlocks).
template <int END>
cudaError_t launch_tokens(const TileArgs& a, int dtype, const CUtensorMap& mp, const CUtensorMap& mq, cudaStream_t stream) {
    return a.splits > 1 ? launch_end<END, kBothMn, true>(a, dtype, pairs_of(a), mp, mq, stream)
                        : launch_end<END, kBothMn>(a, dtype, pairs_of(a), mp, mq, stream);
}

// out [n] from the parts' sums.
cudaError_t sum_up(const float* sums, uint32_t parts, const float* scale, void* out, int64_t n, int dtype, cudaStream_t stream) {
    const int64_t blocks = (n + 2 * entropy::kSumThreads - 1) / (2 * entropy::kSumThreads);
    if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    return launch(dtype == kBF16 ? entropy::sum_kernel<kBF16> : entropy::sum_kernel<kF16>, uint32_t(blocks), entropy::kSumThreads,
                  stream, sums, scale, static_cast<uint16_t*>(out), n, parts);
}

// The tile of rows (a multiple of `step`) that pair_kernel takes, by plan_of's
// estimate of its rounds.
uint32_t pair_width(int64_t N, int64_t M, int64_t kb, int64_t step) {
    uint32_t best = 256;
    int64_t least = INT64_MAX;
    for (int64_t w = 128; w <= 256; w += step) {
        const int64_t rounds = ((N + 255) / 256 * ((M + w - 1) / w) + kPairsAtOnce - 1) / kPairsAtOnce;
        const int64_t cost = 21 * w + rounds * (kb * (41 * w / 20 > 300 ? 41 * w / 20 : 300) + 1500);
        if (cost < least) least = cost, best = uint32_t(w);
    }
    return best;
}

}  // namespace

int64_t entropy_pairs(int64_t T, int64_t V) {
    const int64_t group = T <= kFewRows ? kEntropyUnit : entropy_group(V);
    return T * ((V + group - 1) / group);
}

namespace {

// The logits' sums over the runs of K, tiles of their own, in FP32: [runs,T,V].
cudaError_t apart_sums(const EntropyCall& c, uint32_t runs, float* sums) {
    const Product p = {c.x, c.w, c.x_stride, c.w_stride, false, false, true, c.T, c.V, c.I, {}};
    const bool few = c.T <= kFewRows;
    TileArgs a;
    CUtensorMap mp, mq;
    const cudaError_t e = few ? lay_out_few(p, c.dtype, apart_lanes(c.V, runs), runs, a, mp, mq)
                              : lay_out(p, c.dtype, {true, apart_width(c.V, c.T, runs), runs}, a, mp, mq);
    if (e != cudaSuccess) return e;
    a.end = {};
    a.end.sum_out = sums;
    static std::atomic<uint64_t> allowed{0};
    return few ? launch_few<false, kBF16, kEndSum>(a, mp, mq, c.stream)
               : launch_pair_kernel(pair_kernel<false, kBF16, kBothK, false, kEndSum>, allowed, a, pairs_of(a, runs), mp, mq, c.stream);
}

}  // namespace

cudaError_t entropy_fwd_apart(const EntropyCall& c, float* loss, float* lse, float* sums) {
    const uint32_t runs = entropy_runs((c.I + 63) / 64);
    const cudaError_t e = apart_sums(c, runs, sums);
    if (e != cudaSuccess) return e;
    const int64_t units = (c.V + kEntropyUnit - 1) / kEntropyUnit;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(uint32_t(c.T));
    // more tokens than SMs have few entries each (T = 256, V = 1024 13.0 us with 1024 threads, 11.5 with 256)
    const bool wide = c.T <= num_sms();
    cfg.blockDim = dim3(wide ? 1024 : 256);
    cfg.dynamicSmemBytes = size_t(units) * 8;
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, wide ? entropy::apart_join_kernel<1024> : entropy::apart_join_kernel<256>, sums, c.target, loss, lse, c.T, c.V, runs);
}

cudaError_t entropy_fwd(const EntropyCall& c, float* loss, float* lse, float2* partial, float* at) {
    const bool few = c.T <= kFewRows;
    const int64_t group = entropy_group(c.V), units = entropy_pairs(c.T, c.V) / c.T, groups = (c.V + group - 1) / group;
    Product p;   // the vocabulary on the lanes, or, with more tokens, the tokens
    const Product by_entry = {c.x, c.w, c.x_stride, c.w_stride, false, false, true, c.T, c.V, c.I, {}};
    const Product by_token = {c.w, c.x, c.w_stride, c.x_stride, false, false, true, c.V, c.T, c.I, {}};
    p = few ? by_entry : by_token;
    TileArgs a;
    CUtensorMap mp, mq;
    const uint32_t runs = entropy_runs(k_blocks(p, c.dtype));
    const uint32_t width = group == 64 ? 256 : pair_width(c.T, c.V, k_blocks(p, c.dtype), 128);
    cudaError_t e = few ? lay_out_few(p, c.dtype, few_lanes(c.V), runs, a, mp, mq)
                        : lay_out(p, c.dtype, {true, width, runs}, a, mp, mq);
    if (e != cudaSuccess) return e;
    a.end = {};
    a.end.partial = partial, a.end.units = units, a.end.group = uint32_t(group), a.end.at = at, a.end.target = c.target;
    static std::atomic<uint64_t> allowed{0};
    e = few ? launch_few<false, kBF16, kEndEntropy>(a, mp, mq, c.stream)
            : launch_pair_kernel(pair_kernel<false, kBF16, kBothK, false, kEndEntropy>, allowed, a, pairs_of(a), mp, mq, c.stream);
    if (e != cudaSuccess) return e;
    const bool wide = groups > entropy::kJoinGroups;
    const int64_t per_block = wide ? 1 : entropy::kJoinThreads / 32;
    constexpr int kWide = entropy::kJoinThreads;
    auto* join = few ? (wide ? entropy::join_kernel<kWide, 4> : entropy::join_kernel<32, 4>)
                     : (wide ? entropy::join_kernel<kWide, 1> : entropy::join_kernel<32, 1>);
    return launch(join,
                  uint32_t((c.T + per_block - 1) / per_block), entropy::kJoinThreads, c.stream, partial, at, c.target, loss, lse, c.T,
                  c.V, units, few ? uint32_t(group / kEntropyUnit) : 1u);
}

// d [T,count] with the tokens on the lanes: a thread has the entries of one token.
cudaError_t entropy_logit_grad(const EntropyCall& c, const EntropyGrads& g, const float* lse, int64_t first, int64_t count,
                               uint16_t* d, int64_t pitch) {
    const void* w = static_cast<const uint16_t*>(c.w) + first * c.w_stride;
    Product p = {w, c.x, c.w_stride, c.x_stride, false, false, false, count, c.T, c.I, {}};
    p.e.y = d;
    TileArgs a;
    CUtensorMap mp, mq;
    const cudaError_t e = lay_out(p, c.dtype, {true, pair_width(c.T, count, k_blocks(p, c.dtype), 32), 1}, a, mp, mq);
    if (e != cudaSuccess) return e;
    a.end = {};
    a.end.inverse = g.inverse, a.end.target = c.target, a.end.lse = lse, a.end.grad_loss = g.loss, a.end.grad_lse = g.lse;
    a.end.first = first, a.end.entries = c.V, a.end.pitch = pitch;
    return launch_end<kEndProb, kBothK>(a, c.dtype, pairs_of(a), mp, mq, c.stream);
}

cudaError_t entropy_logit_grad_apart(const EntropyCall& c, const EntropyGrads& g, const float* lse, float* sums, uint16_t* d,
                                     int64_t pitch) {
    const uint32_t runs = entropy_runs((c.I + 63) / 64);
    const cudaError_t e = apart_sums(c, runs, sums);
    if (e != cudaSuccess) return e;
    TileArgs a = {};
    a.e.y = d;
    a.rows = uint32_t(c.T);
    a.end.inverse = g.inverse, a.end.target = c.target, a.end.lse = lse, a.end.grad_loss = g.loss, a.end.grad_lse = g.lse;
    a.end.entries = c.V, a.end.pitch = pitch;
    const uint32_t by_token = uint32_t((c.V + 2 * entropy::kApartGradThreads - 1) / (2 * entropy::kApartGradThreads));
    return launch(c.dtype == kBF16 ? entropy::apart_grad_kernel<kBF16> : entropy::apart_grad_kernel<kF16>, uint32_t(c.T) * by_token,
                  entropy::kApartGradThreads, c.stream, sums, a, c.V, runs, by_token);
}

uint32_t entropy_parts(int64_t T, int64_t I, int64_t count) { return sum_plan(I, T, (count + 63) / 64).splits; }

cudaError_t entropy_grad_x(const EntropyCall& c, const uint16_t* d, int64_t pitch, int64_t first, int64_t count, uint32_t parts,
                           const float* sum_in, float* sum_out, const float* scale, void* grad_x) {
    const void* w = static_cast<const uint16_t*>(c.w) + first * c.w_stride;
    Product p = {d, w, pitch, c.w_stride, false, true, false, c.T, c.I, count, {}};   // [T,I] = d [T,count] . w[first ..] [count,I]
    p.e.y = static_cast<uint16_t*>(grad_x);
    const int64_t kb = k_blocks(p, c.dtype);
    Plan plan = sum_plan(c.I, c.T, kb);
    plan.splits = kb < parts ? uint32_t(kb) : parts;   // (a last, shorter piece adds to the first of them)
    TileArgs a;
    CUtensorMap mp, mq;
    const cudaError_t e = lay_out(p, c.dtype, plan, a, mp, mq);
    if (e != cudaSuccess) return e;
    a.end = {};
    a.end.sum_in = sum_in, a.end.sum_out = sum_out, a.end.scale = scale;
    return launch_end<kEndSum, kPMnQK>(a, c.dtype, pairs_of(a, a.splits), mp, mq, c.stream);
}

cudaError_t entropy_sum(const EntropyCall& c, const float* sums, uint32_t parts, const float* scale, void* grad_x) {
    return sum_up(sums, parts, scale, grad_x, c.T * c.I, c.dtype, c.stream);
}

// [count,I] = d^T [count,T] . x [T,I].  Where grad_w's rows are whole sectors
// the vocabulary is on the lanes and a thread stores a row's values by sectors;
// rows at any alignment have their values on the lanes (I = 1279: 153 us of a
// call that took 483 by rows).
cudaError_t entropy_grad_w(const EntropyCall& c, const uint16_t* d, int64_t pitch, int64_t first, int64_t count,
                           const float* scale, void* grad_w) {
    uint16_t* out = static_cast<uint16_t*>(grad_w) + first * c.I;
    Product p = {d, c.x, pitch, c.x_stride, true, true, false, count, c.I, c.T, {}};
    p.e.y = out;
    if (c.I % 16 == 0 && aligned(out, 32)) return row_product(p, scale, c.dtype, c.stream);
    TileArgs a;
    CUtensorMap mp, mq;
    const int64_t kb = k_blocks(p, c.dtype);
    const cudaError_t e = lay_out(p, c.dtype, {true, pair_width(p.N, p.M, kb, 128), sum_parts(kb)}, a, mp, mq);
    if (e != cudaSuccess) return e;
    a.end = {};
    a.end.scale = scale;
    return launch_tokens<kEndSum>(a, c.dtype, mp, mq, c.stream);
}

cudaError_t row_product(const Product& p, const float* scale, int dtype, cudaStream_t stream) {
    // the product's transpose, with the output's rows on the lanes
    Product t = {p.b, p.a, p.b_stride, p.a_stride, true, true, false, p.N, p.M, p.K, {}};
    t.e.y = p.e.y;
    TileArgs a;
    CUtensorMap mp, mq;
    const int64_t kb = k_blocks(t, dtype);
    const cudaError_t e = lay_out(t, dtype, {true, pair_width(t.N, t.M, kb, 128), sum_parts(kb)}, a, mp, mq);
    if (e != cudaSuccess) return e;
    a.end = {};
    a.end.scale = scale, a.end.pitch = p.N;
    return launch_tokens<kEndRow>(a, dtype, mp, mq, stream);
}

cudaError_t apart_product(const Product& p, float* sums, int dtype, cudaStream_t stream) {
    TileArgs a;
    CUtensorMap mp, mq;
    cudaError_t e = lay_out(p, dtype, sum_plan(p.N, p.M, k_blocks(p, dtype), 128), a, mp, mq);
    if (e != cudaSuccess) return e;
    a.end = {};
    a.end.sum_out = sums;
    e = launch_end<kEndSum, kBothMn>(a, dtype, pairs_of(a, a.splits), mp, mq, stream);
    return e == cudaSuccess ? sum_up(sums, a.splits, nullptr, p.e.y, p.M * p.N, dtype, stream) : e;
}

}  // namespace layer
}  // namespace mhc
