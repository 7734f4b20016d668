// C ABI of the layer operators (mhc_layer.h): argument validation and launch
// through mhc_layer_launch.cuh.

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "mhc_layer.h"
#include "mhc_layer_launch.cuh"

namespace mhc {
namespace layer {

int num_sms() {
    static std::atomic<int> cached[kMaxDevices];
    const int dev = current_device();
    if (dev < 0) return 152;
    int n = cached[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 152;
        cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

}  // namespace layer
}  // namespace mhc

namespace {

using mhc::layer::aligned;

constexpr int kAbiVersion = 1;

thread_local int32_t g_last_cuda_error = 0;

mhc_status_t finish(cudaError_t e) {
    if (e != cudaSuccess) cudaGetLastError();   // reported here, not by the next call
    g_last_cuda_error = int32_t(e);
    return e == cudaSuccess ? MHC_OK : MHC_ERR_CUDA;
}

inline cudaStream_t cu(mhc_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

inline bool dtype_ok(int32_t d) { return d == MHC_DTYPE_BF16 || d == MHC_DTYPE_F16; }

// A buffer of a call: its bytes from the first to the last one touched.
// ok is false for a missing, misaligned or too large one.
struct Buffer {
    uintptr_t lo = 0, hi = 0;
    bool ok = true;
};

Buffer rows(const void* p, int64_t count, int64_t length, int64_t stride, int64_t size, bool optional = false) {
    Buffer b;
    if (p == nullptr) {
        b.ok = optional;
        return b;
    }
    if (count < 0 || length < 0 || stride < length || !aligned(p, uintptr_t(size))) {
        b.ok = false;
        return b;
    }
    if (count == 0 || length == 0) return b;
    const int64_t most = (INT64_MAX / size - length) / (count > 1 ? count - 1 : 1);
    if (length > INT64_MAX / size || stride > most) {
        b.ok = false;
        return b;
    }
    b.lo = reinterpret_cast<uintptr_t>(p);
    b.hi = b.lo + uintptr_t(((count - 1) * stride + length) * size);
    b.ok = b.hi >= b.lo;
    return b;
}

inline Buffer dense(const void* p, int64_t count, int64_t length, int64_t size, bool optional = false) {
    return rows(p, count, length, length, size, optional);
}

inline bool apart(const Buffer& a, const Buffer& b) { return a.hi <= b.lo || b.hi <= a.lo; }

// Every buffer is valid and no output touches an input or another output.
template <int NO, int NI>
bool valid(const Buffer (&outs)[NO], const Buffer (&ins)[NI]) {
    for (const Buffer& in : ins)
        if (!in.ok) return false;
    for (int i = 0; i < NO; ++i) {
        if (!outs[i].ok) return false;
        for (int j = i + 1; j < NO; ++j)
            if (!apart(outs[i], outs[j])) return false;
        for (const Buffer& in : ins)
            if (!apart(outs[i], in)) return false;
    }
    return true;
}

inline Buffer workspace_of(const void* p, int64_t bytes, int64_t need) {
    Buffer b;
    if (need == 0) return b;
    b = dense(p, 1, bytes, 1);
    b.ok = b.ok && bytes >= need && aligned(p, 16);
    return b;
}

// ---- RMS norm --------------------------------------------------------------

mhc_status_t norm_fwd(const void* x, const void* residual, const float* weight, void* y, float* scale, void* total,
                      float* rstd, int64_t T, int64_t H, int64_t x_stride, int64_t residual_stride, float eps, int out,
                      int32_t dtype, mhc_stream_t stream) {
    using namespace mhc::norm;
    if (!dtype_ok(dtype) || T < 0 || H <= 0) return MHC_ERR_INVALID_ARG;
    if (H > kMaxH) return MHC_ERR_UNSUPPORTED;
    if (T == 0) return MHC_OK;
    if ((residual == nullptr) != (total == nullptr)) return MHC_ERR_INVALID_ARG;
    const int64_t groups = out == kOutFp8Group ? (H + kGroup - 1) / kGroup : 1;
    const Buffer outs[4] = {dense(y, T, H, out == kOutSame ? 2 : 1), dense(total, T, H, 2, true), dense(rstd, T, 1, 4),
                            dense(scale, T, groups, 4, out == kOutSame)};
    const Buffer ins[3] = {rows(x, T, H, x_stride, 2), rows(residual, T, H, residual_stride, 2, true),
                           dense(weight, 1, H, 4)};
    if (!valid(outs, ins)) return MHC_ERR_INVALID_ARG;
    FwdArgs a;
    a.x = static_cast<const uint16_t*>(x);
    a.residual = static_cast<const uint16_t*>(residual);
    a.weight = weight;
    a.y = y;
    a.scale = scale;
    a.total = static_cast<uint16_t*>(total);
    a.rstd = rstd;
    a.timeouts = nullptr;
    a.T = T;
    a.x_stride = x_stride, a.residual_stride = residual_stride;
    a.H = uint32_t(H);
    a.eps = eps;
    return finish(mhc::layer::norm_fwd(a, dtype, out, cu(stream)));
}

mhc_status_t norm_bwd(const void* g, const void* s, const float* weight, const float* rstd, const void* grad_total,
                      void* grad_x, float* grad_weight, void* workspace, int64_t workspace_bytes, int64_t T, int64_t H,
                      int64_t g_stride, int64_t s_stride, int32_t dtype, mhc_stream_t stream) {
    using namespace mhc::norm;
    if (!dtype_ok(dtype) || T < 0 || H <= 0) return MHC_ERR_INVALID_ARG;
    if (H > kMaxH) return MHC_ERR_UNSUPPORTED;
    if (T == 0) {
        if (!dense(grad_weight, 1, H, 4).ok) return MHC_ERR_INVALID_ARG;
        return finish(cudaMemsetAsync(grad_weight, 0, size_t(H) * 4, cu(stream)));
    }
    const int64_t need = mhc_rms_norm_bwd_workspace(T, H);
    const Buffer outs[3] = {dense(grad_x, T, H, 2), dense(grad_weight, 1, H, 4),
                            workspace_of(workspace, workspace_bytes, need)};
    const Buffer ins[5] = {rows(g, T, H, g_stride, 2), rows(s, T, H, s_stride, 2), dense(weight, 1, H, 4),
                           dense(rstd, T, 1, 4), dense(grad_total, T, H, 2, true)};
    if (!valid(outs, ins)) return MHC_ERR_INVALID_ARG;
    BwdArgs a;
    a.g = static_cast<const uint16_t*>(g);
    a.s = static_cast<const uint16_t*>(s);
    a.weight = weight;
    a.rstd = rstd;
    a.grad_total = static_cast<const uint16_t*>(grad_total);
    a.grad_x = static_cast<uint16_t*>(grad_x);
    a.partial = nullptr;
    a.timeouts = nullptr;
    a.T = T;
    a.g_stride = g_stride, a.s_stride = s_stride;
    a.H = uint32_t(H);
    return finish(mhc::layer::norm_bwd(a, grad_weight, static_cast<float*>(workspace), dtype, cu(stream)));
}

// ---- matrix product ----------------------------------------------------------

constexpr int64_t kMaxSide = int64_t(1) << 30;   // coordinates are 32-bit

inline int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }

// An operand [rows, length] as the product reads it: in place where its rows
// start on 16-byte boundaries, else copied to such rows in the workspace.
struct Operand {
    const void* p;
    int64_t rows, length, stride, size;
    bool in_place;

    Operand(const void* ptr, int64_t r, int64_t l, int64_t s, int64_t sz, bool ptr_aligned)
        : p(ptr), rows(r), length(l), stride(s), size(sz), in_place(ptr_aligned && (s * sz % 16 == 0 || r <= 1)) {}
    // 2-byte rows start on sectors of 32 bytes (T = 4096, 4096 -> 7160 backwards with silu 314
    // us, rows of 16 bytes 320)
    int64_t pitch() const { return round16(length); }
    int64_t bytes() const { return in_place ? 0 : rows * pitch() * size; }
    // Gives the operand its place at `at` if it needs one, and moves `at` past it.
    void place(char*& at, mhc::layer::RepackCall* calls, int& count) {
        if (in_place) return;
        calls[count++] = {p, at, rows, length * size, stride * size, pitch() * size};
        p = at, stride = pitch(), in_place = true;
        at += rows * stride * size;
    }
};

inline bool act_ok(int32_t a) { return a >= MHC_ACT_NONE && a <= MHC_ACT_GELU; }

mhc_status_t linear_fwd(const void* x, const float* x_scale, const void* w, const float* w_scale, const float* bias,
                        const void* residual, void* y, void* preact, void* workspace, int64_t workspace_bytes,
                        int64_t T, int64_t I, int64_t O, int64_t x_stride, int64_t w_stride, int64_t residual_stride,
                        int32_t act, bool fp8, int32_t dtype, mhc_stream_t stream) {
    if (!dtype_ok(dtype) || !act_ok(act) || T < 0 || I <= 0 || O <= 0) return MHC_ERR_INVALID_ARG;
    if (T > kMaxSide || I > kMaxSide || O > kMaxSide) return MHC_ERR_UNSUPPORTED;
    if (T == 0) return MHC_OK;
    const int64_t size = fp8 ? 1 : 2;
    Operand a(x, T, I, x_stride, size, aligned(x, 16)), b(w, O, I, w_stride, size, aligned(w, 16));
    const int64_t need = a.bytes() + b.bytes();
    const Buffer outs[3] = {dense(y, T, O, 2), dense(preact, T, O, 2, true),
                            workspace_of(workspace, workspace_bytes, need)};
    const Buffer ins[6] = {rows(x, T, I, x_stride, size), rows(w, O, I, w_stride, size),
                           dense(x_scale, T, 1, 4, !fp8), dense(w_scale, O, 1, 4, !fp8), dense(bias, O, 1, 4, true),
                           rows(residual, T, O, residual_stride, 2, true)};
    if (!valid(outs, ins)) return MHC_ERR_INVALID_ARG;
    char* at = static_cast<char*>(workspace);
    mhc::layer::RepackCall calls[2];
    int count = 0;
    a.place(at, calls, count);
    b.place(at, calls, count);
    if (count > 0) {
        const cudaError_t e = mhc::layer::repack(calls, count, cu(stream));
        if (e != cudaSuccess) return finish(e);
    }
    mhc::linear::Product p;
    p.a = a.p, p.b = b.p;
    p.a_stride = a.stride, p.a_mn = false, p.b_stride = b.stride, p.b_mn = false;
    p.by_row = true;
    p.M = T, p.N = O, p.K = I;
    p.e = {fp8 ? x_scale : nullptr, fp8 ? w_scale : nullptr, bias, static_cast<const uint16_t*>(residual),
           static_cast<uint16_t*>(y), static_cast<uint16_t*>(preact), residual_stride, int(act)};
    return finish(mhc::layer::product(p, fp8 ? mhc::linear::kE4m3 : int(dtype), dtype, cu(stream)));
}

}  // namespace

extern "C" {

int32_t mhc_layer_abi_version(void) { return kAbiVersion; }

int32_t mhc_layer_last_cuda_error(void) { return g_last_cuda_error; }

int64_t mhc_layer_wait_timeouts(void) { return mhc::layer::take_wait_timeouts(); }

mhc_status_t mhc_rms_norm_fwd(const void* x, const void* residual, const float* weight, void* y, void* total,
                              float* rstd, int64_t T, int64_t H, int64_t x_stride, int64_t residual_stride, float eps,
                              mhc_dtype_t dtype, mhc_stream_t stream) {
    return norm_fwd(x, residual, weight, y, nullptr, total, rstd, T, H, x_stride, residual_stride, eps,
                    mhc::norm::kOutSame, dtype, stream);
}

mhc_status_t mhc_rms_norm_fp8_fwd(const void* x, const void* residual, const float* weight, void* y8, float* scale,
                                  void* total, float* rstd, int64_t T, int64_t H, int64_t x_stride,
                                  int64_t residual_stride, float eps, int32_t group, mhc_dtype_t dtype,
                                  mhc_stream_t stream) {
    if (group != 0 && group != mhc::norm::kGroup) return MHC_ERR_UNSUPPORTED;
    return norm_fwd(x, residual, weight, y8, scale, total, rstd, T, H, x_stride, residual_stride, eps,
                    group == 0 ? mhc::norm::kOutFp8Row : mhc::norm::kOutFp8Group, dtype, stream);
}

int64_t mhc_rms_norm_bwd_workspace(int64_t T, int64_t H) {
    if (T <= 0 || H <= 0 || H > mhc::norm::kMaxH || mhc::layer::norm_bwd_partials(T, H) <= 1) return 0;
    return int64_t(mhc::layer::norm_bwd_partials(T, H)) * ((H + 7) / 8 * 8) * 4;
}

mhc_status_t mhc_rms_norm_bwd(const void* g, const void* s, const float* weight, const float* rstd,
                              const void* grad_total, void* grad_x, float* grad_weight, void* workspace,
                              int64_t workspace_bytes, int64_t T, int64_t H, int64_t g_stride, int64_t s_stride,
                              mhc_dtype_t dtype, mhc_stream_t stream) {
    return norm_bwd(g, s, weight, rstd, grad_total, grad_x, grad_weight, workspace, workspace_bytes, T, H, g_stride,
                    s_stride, dtype, stream);
}

int64_t mhc_linear_workspace(int64_t T, int64_t I, int64_t O, int64_t x_stride, int64_t w_stride, int32_t itemsize,
                             int32_t aligned) {
    if (T <= 0 || I <= 0 || O <= 0 || (itemsize != 1 && itemsize != 2)) return 0;
    return Operand(nullptr, T, I, x_stride, itemsize, aligned != 0).bytes() +
           Operand(nullptr, O, I, w_stride, itemsize, aligned != 0).bytes();
}

mhc_status_t mhc_linear_fwd(const void* x, const void* w, const float* bias, const void* residual, void* y,
                            void* preact, void* workspace, int64_t workspace_bytes, int64_t T, int64_t I, int64_t O,
                            int64_t x_stride, int64_t w_stride, int64_t residual_stride, mhc_activation_t act,
                            mhc_dtype_t dtype, mhc_stream_t stream) {
    return linear_fwd(x, nullptr, w, nullptr, bias, residual, y, preact, workspace, workspace_bytes, T, I, O, x_stride,
                      w_stride, residual_stride, act, false, dtype, stream);
}

mhc_status_t mhc_linear_fp8_fwd(const void* x8, const float* x_scale, const void* w8, const float* w_scale,
                                const float* bias, const void* residual, void* y, void* preact, void* workspace,
                                int64_t workspace_bytes, int64_t T, int64_t I, int64_t O, int64_t x_stride,
                                int64_t w_stride, int64_t residual_stride, mhc_activation_t act, mhc_dtype_t dtype,
                                mhc_stream_t stream) {
    return linear_fwd(x8, x_scale, w8, w_scale, bias, residual, y, preact, workspace, workspace_bytes, T, I, O,
                      x_stride, w_stride, residual_stride, act, true, dtype, stream);
}

// The workspace of the backward: u with rows on 16-byte boundaries, where it
// is not g itself, the column sums of the bias gradient, then the operands
// that have to be laid out again.
static int64_t bwd_workspace(int64_t T, int64_t I, int64_t O, int32_t act, bool want_x, bool want_w, bool want_bias,
                             bool g_aligned, bool x_aligned, bool w_aligned) {
    const bool want_u = want_x || want_w;
    const int64_t runs = mhc::layer::slope_partials(T);
    int64_t n = want_bias && runs > 1 ? round16(runs * O * 4) : 0;
    if (want_u) n += Operand(nullptr, T, O, O, 2, g_aligned && act == MHC_ACT_NONE).bytes();
    if (want_w) n += Operand(nullptr, T, I, I, 2, x_aligned).bytes();
    if (want_x) n += Operand(nullptr, O, I, I, 2, w_aligned).bytes();
    return n;
}

int64_t mhc_linear_bwd_workspace(int64_t T, int64_t I, int64_t O, mhc_activation_t act, int32_t want_x, int32_t want_w,
                                 int32_t want_bias, int32_t aligned) {
    if (T <= 0 || I <= 0 || O <= 0) return 0;
    const bool al = aligned != 0;
    return bwd_workspace(T, I, O, act, want_x != 0, want_w != 0, want_bias != 0, al, al, al);
}

mhc_status_t mhc_linear_bwd(const void* g, const void* x, const void* w, const void* preact, void* grad_x,
                            void* grad_w, float* grad_bias, void* workspace, int64_t workspace_bytes, int64_t T,
                            int64_t I, int64_t O, mhc_activation_t act, mhc_dtype_t dtype, mhc_stream_t stream) {
    if (!dtype_ok(dtype) || !act_ok(act) || T < 0 || I <= 0 || O <= 0) return MHC_ERR_INVALID_ARG;
    if (T > kMaxSide || I > kMaxSide || O > kMaxSide) return MHC_ERR_UNSUPPORTED;
    if (T == 0) {
        const Buffer outs[2] = {dense(grad_w, O, I, 2, true), dense(grad_bias, O, 1, 4, true)};
        if (!outs[0].ok || !outs[1].ok) return MHC_ERR_INVALID_ARG;
        cudaError_t e = cudaSuccess;
        if (grad_w != nullptr) e = cudaMemsetAsync(grad_w, 0, size_t(O) * I * 2, cu(stream));
        if (e == cudaSuccess && grad_bias != nullptr) e = cudaMemsetAsync(grad_bias, 0, size_t(O) * 4, cu(stream));
        return finish(e);
    }
    const bool want_x = grad_x != nullptr, want_w = grad_w != nullptr;
    const int64_t need = bwd_workspace(T, I, O, act, want_x, want_w, grad_bias != nullptr, aligned(g, 16), aligned(x, 16),
                                       aligned(w, 16));
    const Buffer outs[4] = {dense(grad_x, T, I, 2, true), dense(grad_w, O, I, 2, true), dense(grad_bias, O, 1, 4, true),
                            workspace_of(workspace, workspace_bytes, need)};
    const Buffer ins[4] = {dense(g, T, O, 2), dense(x, T, I, 2, !want_w), dense(w, O, I, 2, !want_x),
                           dense(preact, T, O, 2, act == MHC_ACT_NONE)};
    if (!valid(outs, ins)) return MHC_ERR_INVALID_ARG;
    char* at = static_cast<char*>(workspace);
    float* partial = reinterpret_cast<float*>(at);
    const int64_t runs = mhc::layer::slope_partials(T);
    if (grad_bias != nullptr && runs > 1) at += round16(runs * O * 4);
    cudaError_t e = cudaSuccess;
    Operand u(g, T, O, O, 2, aligned(g, 16) && act == MHC_ACT_NONE);
    uint16_t* own = act != MHC_ACT_NONE && (want_x || want_w) ? reinterpret_cast<uint16_t*>(at) : nullptr;
    if (own != nullptr) {
        at += u.bytes();
        u.p = own, u.stride = u.pitch(), u.in_place = true;
    }
    Operand xo(x, T, I, I, 2, aligned(x, 16)), wo(w, O, I, I, 2, aligned(w, 16));
    mhc::layer::RepackCall calls[3];
    int count = 0;
    if (want_x || want_w) u.place(at, calls, count);
    if (want_w) xo.place(at, calls, count);
    if (want_x) wo.place(at, calls, count);
    for (int i = 0; i < count; i += 2) {
        e = mhc::layer::repack(calls + i, count - i < 2 ? 1 : 2, cu(stream));
        if (e != cudaSuccess) return finish(e);
    }
    mhc::linear::Product p;
    if (act != MHC_ACT_NONE || grad_bias != nullptr) {
        e = mhc::layer::slope(static_cast<const uint16_t*>(g),
                              act == MHC_ACT_NONE ? nullptr : static_cast<const uint16_t*>(preact), own, grad_bias,
                              partial, T, O, u.pitch(), int(act), dtype, cu(stream));
        if (e != cudaSuccess) return finish(e);
    }
    p.e = {nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, mhc::linear::kActNone};
    if (want_x) {   // [T,I] = u [T,O] . w [O,I]
        p.a = u.p, p.a_stride = u.stride, p.a_mn = false;
        p.b = wo.p, p.b_stride = wo.stride, p.b_mn = true;
        p.M = T, p.N = I, p.K = O, p.by_row = true;
        p.e.y = static_cast<uint16_t*>(grad_x);
        e = mhc::layer::product(p, dtype, dtype, cu(stream));
        if (e != cudaSuccess) return finish(e);
    }
    if (want_w) {   // [O,I] = u^T [O,T] . x [T,I]
        p.a = u.p, p.a_stride = u.stride, p.a_mn = true;
        p.b = xo.p, p.b_stride = xo.stride, p.b_mn = true;
        p.M = O, p.N = I, p.K = T, p.by_row = false;
        p.e.y = static_cast<uint16_t*>(grad_w);
        e = mhc::layer::product(p, dtype, dtype, cu(stream));
        if (e != cudaSuccess) return finish(e);
    }
    return finish(cudaSuccess);
}

mhc_status_t mhc_rotary(const void* x, const int64_t* positions, const float* frequencies, void* out, int64_t T,
                        int64_t heads, int64_t D, int64_t R, int64_t x_token, int64_t x_head, int64_t out_token,
                        int64_t out_head, float magnitude, int32_t interleaved, int32_t inverse, mhc_dtype_t dtype,
                        mhc_stream_t stream) {
    if (!dtype_ok(dtype) || T < 0 || heads < 0 || D < 0 || R < 0 || R > D || R % 2 != 0) return MHC_ERR_INVALID_ARG;
    if (D > 65536 || heads > 65536) return MHC_ERR_UNSUPPORTED;
    if (T == 0 || heads == 0 || D == 0) return MHC_OK;
    // a head's span, then a token's; x may also hold a head's tokens inside the head's stride
    if (x_head < D || out_head < D || x_head > INT64_MAX / 2 / heads || out_head > INT64_MAX / 2 / heads)
        return MHC_ERR_INVALID_ARG;
    const int64_t x_row = (heads - 1) * x_head + D, out_row = (heads - 1) * out_head + D;
    const bool by_head = x_token < x_row;
    if (by_head && (x_token < D || x_token > INT64_MAX / 2 / T)) return MHC_ERR_INVALID_ARG;
    const Buffer outs[1] = {rows(out, T, out_row, out_token, 2)};
    const bool in_place = x == out && x_token == out_token && x_head == out_head;
    const Buffer bx = by_head ? rows(x, heads, (T - 1) * x_token + D, x_head, 2) : rows(x, T, x_row, x_token, 2);
    const Buffer ins[3] = {in_place ? Buffer() : bx, dense(positions, T, 1, 8, R == 0),
                           dense(frequencies, 1, R / 2, 4, R == 0)};
    if (!bx.ok || !valid(outs, ins)) return MHC_ERR_INVALID_ARG;
    mhc::layer::RotaryCall c;
    c.x = static_cast<const uint16_t*>(x);
    c.out = static_cast<uint16_t*>(out);
    c.positions = positions, c.frequencies = frequencies;
    c.T = T, c.heads = heads, c.D = D, c.R = R;
    c.x_token = x_token, c.x_head = x_head, c.out_token = out_token, c.out_head = out_head;
    c.magnitude = magnitude;
    c.interleaved = interleaved != 0, c.inverse = inverse != 0;
    c.dtype = dtype;
    c.stream = cu(stream);
    return finish(mhc::layer::rotary(c));
}

}  // extern "C"
