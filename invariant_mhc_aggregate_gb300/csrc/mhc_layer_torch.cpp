// The layer operators' calls from PyTorch without the interpreter's part: for
// arguments of the expected kind (CUDA tensors of the right types, shapes and
// strides) a call here allocates the outputs, takes the current stream and
// enters the C ABI of mhc_layer.h; for anything else it returns None, and
// layer.py checks the arguments one by one and says what is wrong.  A decoded
// token's norm takes 15 us of host time through ctypes and torch.empty, and
// less than 3 us on the GPU.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/Exception.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mhc_layer.h"

namespace {

// A plain CUDA tensor, or null.
const at::Tensor* cuda_tensor(PyObject* o) {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    return t.is_cuda() && t.layout() == at::kStrided ? &t : nullptr;
}

inline int storage(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kBFloat16: return MHC_DTYPE_BF16;
        case at::kHalf: return MHC_DTYPE_F16;
        default: return -1;
    }
}

// [rows, length] of `type` on `device` with contiguous rows; `stride` gets
// the distance between rows.
bool rows_of(const at::Tensor& t, at::ScalarType type, int64_t rows, int64_t length, at::Device device, int64_t& stride) {
    if (t.scalar_type() != type || t.dim() != 2 || t.size(0) != rows || t.size(1) != length || t.device() != device)
        return false;
    if (t.stride(1) != 1 && length > 1) return false;
    stride = rows > 1 ? t.stride(0) : length;
    return stride >= length;
}

bool flat(const at::Tensor& t, at::ScalarType type, int64_t n, at::Device device) {
    return t.scalar_type() == type && t.numel() == n && (t.dim() == 1 || (t.dim() == 2 && t.size(1) == 1)) &&
           t.device() == device && t.is_contiguous();
}

// An optional tensor argument: true if it is None (p stays null) or a tensor.
bool optional(PyObject* o, const at::Tensor*& p) {
    if (o == Py_None) return true;
    p = cuda_tensor(o);
    return p != nullptr;
}

inline at::Tensor empty(at::IntArrayRef size, at::ScalarType type, at::Device device) {
    return at::detail::empty_cuda(size, type, device, std::nullopt);
}

inline void* ptr(const at::Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }

inline mhc_stream_t current(at::Device d) {
    return reinterpret_cast<mhc_stream_t>(c10::cuda::getCurrentCUDAStream(d.index()).stream());
}

PyObject* none() { Py_RETURN_NONE; }

// Wraps n results; a null one becomes None.
PyObject* pack(std::initializer_list<const at::Tensor*> list) {
    PyObject* out = PyTuple_New(Py_ssize_t(list.size()));
    if (out == nullptr) return nullptr;
    Py_ssize_t i = 0;
    for (const at::Tensor* t : list) {
        PyObject* o;
        if (t == nullptr || !t->defined()) {
            Py_INCREF(Py_None);
            o = Py_None;
        } else {
            o = THPVariable_Wrap(*t);
        }
        if (o == nullptr) {
            Py_DECREF(out);
            return nullptr;
        }
        PyTuple_SET_ITEM(out, i++, o);
    }
    return out;
}

// No C++ exception leaves a function that the interpreter called.  Where memory
// runs out the call is declined: layer.py's own allocation then raises torch's
// error for that, which a caller may catch (or succeeds).
template <class F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const c10::OutOfMemoryError&) {
        return none();
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// rms_norm(x, weight, residual, eps, group): group -1 for the 16-bit output.
// (y, scale, total, rstd)
PyObject* rms_norm(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    if (nargs != 5) return none();
    return guarded([&]() -> PyObject* {
        const at::Tensor *x = cuda_tensor(args[0]), *w = cuda_tensor(args[1]), *r = nullptr;
        const double eps = PyFloat_Check(args[3]) ? PyFloat_AS_DOUBLE(args[3]) : -1.0;
        const long group = PyLong_AsLong(args[4]);
        if (x == nullptr || w == nullptr || !optional(args[2], r) || eps < 0 || PyErr_Occurred() || x->dim() != 2) {
            PyErr_Clear();
            return none();
        }
        const int dt = storage(*x);
        const int64_t T = x->size(0), H = x->size(1);
        const at::Device dev = x->device();
        int64_t xs, rs = H;
        if (dt < 0 || !rows_of(*x, x->scalar_type(), T, H, dev, xs) || w->dim() != 1 || !flat(*w, at::kFloat, H, dev) ||
            (r != nullptr && !rows_of(*r, x->scalar_type(), T, H, dev, rs)))
            return none();
        const c10::cuda::CUDAGuard guard(dev);
        at::Tensor y = empty({T, H}, group < 0 ? x->scalar_type() : at::kFloat8_e4m3fn, dev), scale, total;
        if (group >= 0) scale = empty({T, group == 0 ? 1 : (H + 127) / 128}, at::kFloat, dev);
        if (r != nullptr) total = empty({T, H}, x->scalar_type(), dev);
        at::Tensor rstd = empty({T}, at::kFloat, dev);
        void* tp = r != nullptr ? total.data_ptr() : nullptr;
        const mhc_status_t st =
            group < 0 ? mhc_rms_norm_fwd(x->data_ptr(), ptr(r), w->data_ptr<float>(), y.data_ptr(), tp,
                                         rstd.data_ptr<float>(), T, H, xs, rs, float(eps), mhc_dtype_t(dt), current(dev))
                      : mhc_rms_norm_fp8_fwd(x->data_ptr(), ptr(r), w->data_ptr<float>(), y.data_ptr(),
                                             scale.data_ptr<float>(), tp, rstd.data_ptr<float>(), T, H, xs, rs,
                                             float(eps), int32_t(group), mhc_dtype_t(dt), current(dev));
        if (st != MHC_OK) return none();
        return pack({&y, &scale, r != nullptr ? &total : x, &rstd});
    });
}

// rms_norm_backward(grad_y, total, weight, rstd, grad_total) -> (grad_x, grad_weight)
PyObject* rms_norm_backward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    if (nargs != 5) return none();
    return guarded([&]() -> PyObject* {
        const at::Tensor *g = cuda_tensor(args[0]), *s = cuda_tensor(args[1]), *w = cuda_tensor(args[2]),
                         *rstd = cuda_tensor(args[3]), *gt = nullptr;
        if (!g || !s || !w || !rstd || !optional(args[4], gt) || s->dim() != 2) return none();
        const int dt = storage(*s);
        const int64_t T = s->size(0), H = s->size(1);
        const at::Device dev = s->device();
        int64_t gs, ss, ts;
        if (dt < 0 || !rows_of(*s, s->scalar_type(), T, H, dev, ss) || !rows_of(*g, s->scalar_type(), T, H, dev, gs) ||
            w->dim() != 1 || !flat(*w, at::kFloat, H, dev) || rstd->dim() != 1 || !flat(*rstd, at::kFloat, T, dev) ||
            (gt != nullptr && (!rows_of(*gt, s->scalar_type(), T, H, dev, ts) || ts != H)))
            return none();
        const c10::cuda::CUDAGuard guard(dev);
        at::Tensor gx = empty({T, H}, s->scalar_type(), dev), gw = empty({H}, at::kFloat, dev), ws;
        const int64_t need = mhc_rms_norm_bwd_workspace(T, H);
        if (need > 0) ws = empty({need}, at::kByte, dev);
        const mhc_status_t st = mhc_rms_norm_bwd(g->data_ptr(), s->data_ptr(), w->data_ptr<float>(),
                                                 rstd->data_ptr<float>(), ptr(gt), gx.data_ptr(), gw.data_ptr<float>(),
                                                 need > 0 ? ws.data_ptr() : nullptr, need, T, H, gs, ss,
                                                 mhc_dtype_t(dt), current(dev));
        return st == MHC_OK ? pack({&gx, &gw}) : none();
    });
}

// linear(x, x_scale, w, w_scale, bias, act, residual, out_type, keep) ->
// (y, z); out_type: 0 BF16, 1 binary16, -1 that of x; the scales are None
// without E4M3.
PyObject* linear(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    if (nargs != 9) return none();
    return guarded([&]() -> PyObject* {
        const at::Tensor *x = cuda_tensor(args[0]), *sx = nullptr, *w = cuda_tensor(args[2]), *sw = nullptr, *b = nullptr,
                         *r = nullptr;
        if (!x || !w || !optional(args[1], sx) || !optional(args[3], sw) || !optional(args[4], b) ||
            !optional(args[6], r) || x->dim() != 2 || w->dim() != 2 || (sx == nullptr) != (sw == nullptr))
            return none();
        const long act = PyLong_AsLong(args[5]);
        long out = PyLong_AsLong(args[7]);
        const bool keep = args[8] == Py_True, fp8 = sx != nullptr;
        if (PyErr_Occurred()) {
            PyErr_Clear();
            return none();
        }
        if (out < 0) out = storage(*x);
        if (out < 0) return none();
        const int64_t T = x->size(0), I = x->size(1), O = w->size(0);
        const at::Device dev = x->device();
        const at::ScalarType type = out == 0 ? at::kBFloat16 : at::kHalf;
        const at::ScalarType operand = fp8 ? at::kFloat8_e4m3fn : type;
        int64_t xs, ws, rs = O;
        if (!rows_of(*x, operand, T, I, dev, xs) || !rows_of(*w, operand, O, I, dev, ws) ||
            (fp8 && (!flat(*sx, at::kFloat, T, dev) || !flat(*sw, at::kFloat, O, dev))) ||
            (b != nullptr && (b->dim() != 1 || !flat(*b, at::kFloat, O, dev))) ||
            (r != nullptr && !rows_of(*r, type, T, O, dev, rs)))
            return none();
        const c10::cuda::CUDAGuard guard(dev);
        at::Tensor y = empty({T, O}, type, dev), z, work;
        if (keep) z = empty({T, O}, type, dev);
        void *xp = x->data_ptr(), *wp = w->data_ptr();
        const bool aligned = ((reinterpret_cast<uintptr_t>(xp) | reinterpret_cast<uintptr_t>(wp)) & 15) == 0;
        const int64_t need = mhc_linear_workspace(T, I, O, xs, ws, fp8 ? 1 : 2, aligned);
        if (need > 0) work = empty({need}, at::kByte, dev);
        void* workp = need > 0 ? work.data_ptr() : nullptr;
        void* zp = keep ? z.data_ptr() : nullptr;
        const float* bp = b == nullptr ? nullptr : b->data_ptr<float>();
        const mhc_status_t st =
            fp8 ? mhc_linear_fp8_fwd(xp, sx->data_ptr<float>(), wp, sw->data_ptr<float>(), bp, ptr(r), y.data_ptr(), zp,
                                     workp, need, T, I, O, xs, ws, rs, mhc_activation_t(act), mhc_dtype_t(out),
                                     current(dev))
                : mhc_linear_fwd(xp, wp, bp, ptr(r), y.data_ptr(), zp, workp, need, T, I, O, xs, ws, rs,
                                 mhc_activation_t(act), mhc_dtype_t(out), current(dev));
        return st == MHC_OK ? pack({&y, &z}) : none();
    });
}

// linear_backward(grad_y, x, w, z, act, bias, want_x, want_w) -> (grad_x, grad_w, grad_b)
PyObject* linear_backward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    if (nargs != 8) return none();
    return guarded([&]() -> PyObject* {
        const at::Tensor *g = cuda_tensor(args[0]), *x = cuda_tensor(args[1]), *w = cuda_tensor(args[2]), *z = nullptr;
        if (!g || !x || !w || !optional(args[3], z) || x->dim() != 2 || w->dim() != 2) return none();
        const long act = PyLong_AsLong(args[4]);
        const int bias = PyObject_IsTrue(args[5]), want_x = PyObject_IsTrue(args[6]), want_w = PyObject_IsTrue(args[7]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            return none();
        }
        const int dt = storage(*x);
        const int64_t T = x->size(0), I = x->size(1), O = w->size(0);
        const at::Device dev = x->device();
        const at::ScalarType type = x->scalar_type();
        int64_t s;
        if (dt < 0 || !rows_of(*x, type, T, I, dev, s) || s != I || !rows_of(*w, type, O, I, dev, s) || s != I ||
            !rows_of(*g, type, T, O, dev, s) || s != O)
            return none();
        if (act == MHC_ACT_NONE) z = nullptr;
        else if (z == nullptr || !rows_of(*z, type, T, O, dev, s) || s != O) return none();
        const c10::cuda::CUDAGuard guard(dev);
        at::Tensor gx, gw, gb, work;
        if (want_x) gx = empty({T, I}, type, dev);
        if (want_w) gw = empty({O, I}, type, dev);
        if (bias) gb = empty({O}, at::kFloat, dev);
        void *gp = g->data_ptr(), *xp = x->data_ptr(), *wp = w->data_ptr();
        const bool aligned = ((reinterpret_cast<uintptr_t>(gp) | reinterpret_cast<uintptr_t>(xp) |
                               reinterpret_cast<uintptr_t>(wp)) & 15) == 0;
        const int64_t need =
            mhc_linear_bwd_workspace(T, I, O, mhc_activation_t(act), want_x, want_w, bias, aligned);
        if (need > 0) work = empty({need}, at::kByte, dev);
        const mhc_status_t st = mhc_linear_bwd(gp, xp, wp, ptr(z), want_x ? gx.data_ptr() : nullptr,
                                               want_w ? gw.data_ptr() : nullptr, bias ? gb.data_ptr<float>() : nullptr,
                                               need > 0 ? work.data_ptr() : nullptr, need, T, I, O,
                                               mhc_activation_t(act), mhc_dtype_t(dt), current(dev));
        return st == MHC_OK ? pack({&gx, &gw, &gb}) : none();
    });
}

// gated_linear(x, x_scale, w, w_scale, bias, act, out_type, keep) -> (y, z), as linear
PyObject* gated_linear(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    if (nargs != 8) return none();
    return guarded([&]() -> PyObject* {
        const at::Tensor *x = cuda_tensor(args[0]), *sx = nullptr, *w = cuda_tensor(args[2]), *sw = nullptr, *b = nullptr;
        if (!x || !w || !optional(args[1], sx) || !optional(args[3], sw) || !optional(args[4], b) || x->dim() != 2 ||
            w->dim() != 2 || (sx == nullptr) != (sw == nullptr))
            return none();
        const long act = PyLong_AsLong(args[5]);
        long out = PyLong_AsLong(args[6]);
        const bool keep = args[7] == Py_True, fp8 = sx != nullptr;
        if (PyErr_Occurred()) {
            PyErr_Clear();
            return none();
        }
        if (out < 0) out = storage(*x);
        if (out < 0) return none();
        const int64_t T = x->size(0), I = x->size(1), O = w->size(0), F = O / 2;
        const at::Device dev = x->device();
        const at::ScalarType type = out == 0 ? at::kBFloat16 : at::kHalf;
        const at::ScalarType operand = fp8 ? at::kFloat8_e4m3fn : type;
        int64_t xs, ws;
        if (O % 2 != 0 || !rows_of(*x, operand, T, I, dev, xs) || !rows_of(*w, operand, O, I, dev, ws) ||
            (fp8 && (!flat(*sx, at::kFloat, T, dev) || !flat(*sw, at::kFloat, O, dev))) ||
            (b != nullptr && (b->dim() != 1 || !flat(*b, at::kFloat, O, dev))))
            return none();
        const c10::cuda::CUDAGuard guard(dev);
        at::Tensor y = empty({T, F}, type, dev), z, work;
        if (keep) z = empty({T, O}, type, dev);
        void *xp = x->data_ptr(), *wp = w->data_ptr();
        const bool aligned = ((reinterpret_cast<uintptr_t>(xp) | reinterpret_cast<uintptr_t>(wp)) & 15) == 0;
        const int64_t need = mhc_linear_workspace(T, I, O, xs, ws, fp8 ? 1 : 2, aligned);
        if (need > 0) work = empty({need}, at::kByte, dev);
        void* workp = need > 0 ? work.data_ptr() : nullptr;
        void* zp = keep ? z.data_ptr() : nullptr;
        const float* bp = b == nullptr ? nullptr : b->data_ptr<float>();
        const mhc_status_t st =
            fp8 ? mhc_gated_linear_fp8_fwd(xp, sx->data_ptr<float>(), wp, sw->data_ptr<float>(), bp, y.data_ptr(), zp, workp,
                                           need, T, I, F, xs, ws, mhc_activation_t(act), mhc_dtype_t(out), current(dev))
                : mhc_gated_linear_fwd(xp, wp, bp, y.data_ptr(), zp, workp, need, T, I, F, xs, ws, mhc_activation_t(act),
                                       mhc_dtype_t(out), current(dev));
        return st == MHC_OK ? pack({&y, &z}) : none();
    });
}

// gated_linear_backward(grad_y, x, w, z, act, bias, want_x, want_w) -> (grad_x, grad_w, grad_b)
PyObject* gated_linear_backward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    if (nargs != 8) return none();
    return guarded([&]() -> PyObject* {
        const at::Tensor *g = cuda_tensor(args[0]), *x = cuda_tensor(args[1]), *w = cuda_tensor(args[2]), *z = cuda_tensor(args[3]);
        if (!g || !x || !w || !z || x->dim() != 2 || w->dim() != 2) return none();
        const long act = PyLong_AsLong(args[4]);
        const int bias = PyObject_IsTrue(args[5]), want_x = PyObject_IsTrue(args[6]), want_w = PyObject_IsTrue(args[7]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            return none();
        }
        const int dt = storage(*x);
        const int64_t T = x->size(0), I = x->size(1), O = w->size(0), F = O / 2;
        const at::Device dev = x->device();
        const at::ScalarType type = x->scalar_type();
        int64_t xs, ws, s;
        if (dt < 0 || O % 2 != 0 || !rows_of(*x, type, T, I, dev, xs) || !rows_of(*w, type, O, I, dev, ws) ||
            !rows_of(*g, type, T, F, dev, s) || s != F || !rows_of(*z, type, T, O, dev, s) || s != O)
            return none();
        const c10::cuda::CUDAGuard guard(dev);
        at::Tensor gx, gw, gb, work;
        if (want_x) gx = empty({T, I}, type, dev);
        if (want_w) gw = empty({O, I}, type, dev);
        if (bias) gb = empty({O}, at::kFloat, dev);
        void *xp = x->data_ptr(), *wp = w->data_ptr();
        const bool aligned = ((reinterpret_cast<uintptr_t>(xp) | reinterpret_cast<uintptr_t>(wp)) & 15) == 0;
        const int64_t need = mhc_gated_linear_bwd_workspace(T, I, F, xs, ws, want_x, want_w, bias, aligned);
        if (need > 0) work = empty({need}, at::kByte, dev);
        const mhc_status_t st = mhc_gated_linear_bwd(g->data_ptr(), xp, wp, z->data_ptr(), want_x ? gx.data_ptr() : nullptr,
                                                     want_w ? gw.data_ptr() : nullptr, bias ? gb.data_ptr<float>() : nullptr,
                                                     need > 0 ? work.data_ptr() : nullptr, need, T, I, F, xs, ws,
                                                     mhc_activation_t(act), mhc_dtype_t(dt), current(dev));
        return st == MHC_OK ? pack({&gx, &gw, &gb}) : none();
    });
}

// linear_cross_entropy(x, w, target) -> (loss, lse)
PyObject* linear_cross_entropy(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    if (nargs != 3) return none();
    return guarded([&]() -> PyObject* {
        const at::Tensor *x = cuda_tensor(args[0]), *w = cuda_tensor(args[1]), *target = cuda_tensor(args[2]);
        if (!x || !w || !target || x->dim() != 2 || w->dim() != 2 || target->dim() != 1) return none();
        const int dt = storage(*x);
        const int64_t T = x->size(0), I = x->size(1), V = w->size(0);
        const at::Device dev = x->device();
        int64_t xs, ws;
        if (dt < 0 || !rows_of(*x, x->scalar_type(), T, I, dev, xs) || !rows_of(*w, x->scalar_type(), V, I, dev, ws) ||
            !flat(*target, at::kLong, T, dev))
            return none();
        const c10::cuda::CUDAGuard guard(dev);
        at::Tensor loss = empty({T}, at::kFloat, dev), lse = empty({T}, at::kFloat, dev), work;
        void *xp = x->data_ptr(), *wp = w->data_ptr();
        const bool aligned = ((reinterpret_cast<uintptr_t>(xp) | reinterpret_cast<uintptr_t>(wp)) & 15) == 0;
        const int64_t need = mhc_linear_cross_entropy_workspace(T, I, V, xs, ws, aligned);
        if (need > 0) work = empty({need}, at::kByte, dev);
        const mhc_status_t st = mhc_linear_cross_entropy_fwd(xp, wp, target->data_ptr<int64_t>(), loss.data_ptr<float>(),
                                                             lse.data_ptr<float>(), need > 0 ? work.data_ptr() : nullptr, need,
                                                             T, I, V, xs, ws, mhc_dtype_t(dt), current(dev));
        return st == MHC_OK ? pack({&loss, &lse}) : none();
    });
}

// linear_cross_entropy_backward(grad_loss, x, w, target, lse, grad_lse, want_x, want_w) -> (grad_x, grad_w)
PyObject* linear_cross_entropy_backward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    if (nargs != 8) return none();
    return guarded([&]() -> PyObject* {
        const at::Tensor *gl = nullptr, *x = cuda_tensor(args[1]), *w = cuda_tensor(args[2]), *target = cuda_tensor(args[3]),
                         *lse = cuda_tensor(args[4]), *gs = nullptr;
        if (!x || !w || !target || !lse || !optional(args[0], gl) || !optional(args[5], gs) || x->dim() != 2 || w->dim() != 2 ||
            target->dim() != 1 || lse->dim() != 1 || (gl == nullptr && gs == nullptr))
            return none();
        const int want_x = PyObject_IsTrue(args[6]), want_w = PyObject_IsTrue(args[7]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            return none();
        }
        const int dt = storage(*x);
        const int64_t T = x->size(0), I = x->size(1), V = w->size(0);
        const at::Device dev = x->device();
        int64_t xs, ws;
        if (dt < 0 || !rows_of(*x, x->scalar_type(), T, I, dev, xs) || !rows_of(*w, x->scalar_type(), V, I, dev, ws) ||
            !flat(*target, at::kLong, T, dev) || !flat(*lse, at::kFloat, T, dev) ||
            (gl != nullptr && (gl->dim() != 1 || !flat(*gl, at::kFloat, T, dev))) ||
            (gs != nullptr && (gs->dim() != 1 || !flat(*gs, at::kFloat, T, dev))))
            return none();
        const c10::cuda::CUDAGuard guard(dev);
        at::Tensor gx, gw, work;
        if (want_x) gx = empty({T, I}, x->scalar_type(), dev);
        if (want_w) gw = empty({V, I}, x->scalar_type(), dev);
        void *xp = x->data_ptr(), *wp = w->data_ptr();
        const bool aligned = ((reinterpret_cast<uintptr_t>(xp) | reinterpret_cast<uintptr_t>(wp)) & 15) == 0;
        const int64_t need = mhc_linear_cross_entropy_bwd_workspace(T, I, V, xs, ws, want_x, want_w, aligned);
        if (need > 0) work = empty({need}, at::kByte, dev);
        const mhc_status_t st = mhc_linear_cross_entropy_bwd(
            static_cast<const float*>(ptr(gl)), static_cast<const float*>(ptr(gs)), xp, wp, target->data_ptr<int64_t>(),
            lse->data_ptr<float>(), want_x ? gx.data_ptr() : nullptr, want_w ? gw.data_ptr() : nullptr,
            need > 0 ? work.data_ptr() : nullptr, need, T, I, V, xs, ws, mhc_dtype_t(dt), current(dev));
        return st == MHC_OK ? pack({&gx, &gw}) : none();
    });
}

// rotary(x, positions, frequencies, interleaved, scale, inverse) -> (out,)
PyObject* rotary(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    if (nargs != 6) return none();
    return guarded([&]() -> PyObject* {
        const at::Tensor *x = cuda_tensor(args[0]), *p = cuda_tensor(args[1]), *f = cuda_tensor(args[2]);
        const double scale = PyFloat_Check(args[4]) ? PyFloat_AS_DOUBLE(args[4]) : 0.0;
        if (!x || !p || !f || !PyFloat_Check(args[4]) || x->dim() != 3 || p->dim() != 1 || f->dim() != 1) return none();
        const int inter = PyObject_IsTrue(args[3]), inverse = PyObject_IsTrue(args[5]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            return none();
        }
        const int dt = storage(*x);
        const int64_t T = x->size(0), heads = x->size(1), D = x->size(2);
        const at::Device dev = x->device();
        if (dt < 0 || !flat(*p, at::kLong, T, dev) || !flat(*f, at::kFloat, f->numel(), dev) ||
            (x->stride(2) != 1 && D > 1) || heads < 1)
            return none();
        const int64_t head = heads > 1 ? x->stride(1) : D;
        const int64_t token = T > 1 ? x->stride(0) : (heads - 1) * head + D;
        const c10::cuda::CUDAGuard guard(dev);
        at::Tensor out = empty({T, heads, D}, x->scalar_type(), dev);
        const mhc_status_t st = mhc_rotary(x->data_ptr(), p->data_ptr<int64_t>(), f->data_ptr<float>(), out.data_ptr(), T,
                                           heads, D, 2 * f->numel(), token, head, heads * D, D, float(scale), inter,
                                           inverse, mhc_dtype_t(dt), current(dev));
        return st == MHC_OK ? pack({&out}) : none();
    });
}

PyMethodDef methods[] = {
    {"rms_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rms_norm)), METH_FASTCALL, nullptr},
    {"rms_norm_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rms_norm_backward)), METH_FASTCALL, nullptr},
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(linear)), METH_FASTCALL, nullptr},
    {"linear_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(linear_backward)), METH_FASTCALL, nullptr},
    {"gated_linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(gated_linear)), METH_FASTCALL, nullptr},
    {"gated_linear_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(gated_linear_backward)), METH_FASTCALL,
     nullptr},
    {"linear_cross_entropy", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(linear_cross_entropy)), METH_FASTCALL, nullptr},
    {"linear_cross_entropy_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(linear_cross_entropy_backward)),
     METH_FASTCALL, nullptr},
    {"rotary", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rotary)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "mhc_layer_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_mhc_layer_torch(void) { return PyModule_Create(&module); }
