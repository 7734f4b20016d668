"""Python binding of the layer operators in ``include/mhc_layer.h`` (ctypes):
what stands between the mHC aggregate and the mHC post, and the loss at the
model's end.

    y, total, rstd = rms_norm(x, weight, residual=r)             # [T,H]
    y8, scale, total, rstd = rms_norm_fp8(x, weight, residual=r) # E4M3 and its scales
    grad_x, grad_weight = rms_norm_backward(g, total, weight, rstd)

    y = linear(x, w, bias=b, activation="silu", residual=r)      # act(x w^T + b) + r
    y = linear_fp8(x8, x_scale, w8, w_scale, bias=b)
    y, z = linear_preact(x, w, bias=b, activation="silu")        # z for the backward
    grad_x, grad_w, grad_b = linear_backward(g, x, w, z=z, activation="silu")

    h = gated_linear(x, w_gate_up)                               # silu(x w_gate^T) * (x w_up^T), one kernel
    h = gated_linear_fp8(x8, x_scale, w8, w_scale)
    h, z = gated_linear_preact(x, w_gate_up)
    grad_x, grad_w, grad_b = gated_linear_backward(g, x, w_gate_up, z, bias=False)

    loss, lse = linear_cross_entropy(x, w_vocab, target)         # the logits are not kept
    grad_x, grad_w = linear_cross_entropy_backward(grad_loss, x, w_vocab, target, lse)

    q = rotary(q, positions, rotary_frequencies(128))            # [T,heads,D]

As in :mod:`.binding`, this is argument marshalling only: every step runs in
the sm_103a kernels of ``libmhc_layer.so``, there is no fallback, and calls
are asynchronous on ``stream`` (default: the current PyTorch stream of the
tensors' device).  On the current stream the marshalling of valid arguments is
compiled too (``mhc_layer_torch``); the functions here check and name what it
does not take.  Outputs and workspaces are allocated here, on the current
stream; a caller who passes another stream orders the two as with any PyTorch
tensor.  The differentiable forms are in :mod:`.autograd`.
"""

from __future__ import annotations

import ctypes
import importlib.util
import math
import os
import threading

import torch

from . import _build
from .binding import (MHC_DTYPE_BF16, MHC_DTYPE_F16, MHC_ERR_CUDA, MHC_OK)

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}

#: Every symbol include/mhc_layer.h declares, in declaration order.
EXPORTS = (
    "mhc_layer_abi_version",
    "mhc_rms_norm_fwd",
    "mhc_rms_norm_fp8_fwd",
    "mhc_rms_norm_bwd",
    "mhc_rms_norm_bwd_workspace",
    "mhc_linear_fwd",
    "mhc_linear_fp8_fwd",
    "mhc_linear_bwd",
    "mhc_linear_workspace",
    "mhc_linear_bwd_workspace",
    "mhc_gated_linear_fwd",
    "mhc_gated_linear_fp8_fwd",
    "mhc_gated_linear_bwd",
    "mhc_gated_linear_bwd_workspace",
    "mhc_linear_cross_entropy_fwd",
    "mhc_linear_cross_entropy_workspace",
    "mhc_linear_cross_entropy_bwd",
    "mhc_linear_cross_entropy_bwd_workspace",
    "mhc_rotary",
    "mhc_layer_last_cuda_error",
    "mhc_layer_wait_timeouts",
)

_STATUS = {1: "MHC_ERR_INVALID_ARG", 2: "MHC_ERR_UNSUPPORTED", 3: "MHC_ERR_CUDA"}

_lock = threading.Lock()
_lib = None


class LayerError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        text = _STATUS.get(status, f"status {status}")
        if status == MHC_ERR_CUDA:
            text += f" (cudaError {load().mhc_layer_last_cuda_error()})"
        super().__init__(f"{what}: {text}")


def load():
    """Load the compiled library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LAYER_LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build the CUDA libraries first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(path)
        p, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
        for name, res, args in (
                ("mhc_layer_abi_version", i32, []),
                ("mhc_rms_norm_fwd", i32, [p] * 6 + [i64] * 4 + [f32, i32, p]),
                ("mhc_rms_norm_fp8_fwd", i32, [p] * 7 + [i64] * 4 + [f32, i32, i32, p]),
                ("mhc_rms_norm_bwd", i32, [p] * 8 + [i64] * 5 + [i32, p]),
                ("mhc_rms_norm_bwd_workspace", i64, [i64, i64]),
                ("mhc_linear_fwd", i32, [p] * 7 + [i64] * 7 + [i32, i32, p]),
                ("mhc_linear_fp8_fwd", i32, [p] * 9 + [i64] * 7 + [i32, i32, p]),
                ("mhc_linear_bwd", i32, [p] * 8 + [i64] * 4 + [i32, i32, p]),
                ("mhc_linear_workspace", i64, [i64] * 5 + [i32, i32]),
                ("mhc_linear_bwd_workspace", i64, [i64] * 3 + [i32] * 5),
                ("mhc_gated_linear_fwd", i32, [p] * 6 + [i64] * 6 + [i32, i32, p]),
                ("mhc_gated_linear_fp8_fwd", i32, [p] * 8 + [i64] * 6 + [i32, i32, p]),
                ("mhc_gated_linear_bwd", i32, [p] * 8 + [i64] * 6 + [i32, i32, p]),
                ("mhc_gated_linear_bwd_workspace", i64, [i64] * 5 + [i32] * 4),
                ("mhc_linear_cross_entropy_fwd", i32, [p] * 6 + [i64] * 6 + [i32, p]),
                ("mhc_linear_cross_entropy_workspace", i64, [i64] * 5 + [i32]),
                ("mhc_linear_cross_entropy_bwd", i32, [p] * 9 + [i64] * 6 + [i32, p]),
                ("mhc_linear_cross_entropy_bwd_workspace", i64, [i64] * 5 + [i32] * 3),
                ("mhc_rotary", i32, [p] * 4 + [i64] * 8 + [f32, i32, i32, i32, p]),
                ("mhc_layer_last_cuda_error", i32, []),
                ("mhc_layer_wait_timeouts", i64, [])):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
        return lib


_fast = None


def _compiled():
    """The compiled marshalling (raises if it has not been built)."""
    global _fast
    if _fast is None:
        path = _build.TORCH_LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
        spec = importlib.util.spec_from_file_location("mhc_layer_torch", path)
        _fast = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(_fast)
    return _fast


def wait_timeouts() -> int:
    """1 if a bounded wait of the library's kernels ran out on the current
    device since the last call, else 0 (clears it; synchronizes the device);
    -1 on a CUDA error."""
    return int(load().mhc_layer_wait_timeouts())


_DTYPES = {torch.bfloat16: MHC_DTYPE_BF16, torch.float16: MHC_DTYPE_F16}
_E4M3 = torch.float8_e4m3fn

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream, device) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(device.index)
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return int(stream.cuda_stream)
    return int(stream)


def _storage(t: torch.Tensor, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    return code


def _rows(t: torch.Tensor, name: str, dtype, shape, device) -> int:
    """Checks a 2-d tensor of contiguous rows; returns its row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device or device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor on {device}, got {t.device}")
    step, one = t.stride()
    rows, length = shape
    if (one != 1 and length > 1) or (step < length and rows > 1):
        raise ValueError(f"{name} must have contiguous rows that do not overlap, got strides {t.stride()}")
    return step if rows > 1 else length


def _flat(t: torch.Tensor, name: str, dtype, shape, device) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device or device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _two(t: torch.Tensor, name: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-d, got {tuple(t.shape)}")
    return t.shape


def _call(device, name: str, *args) -> None:
    """The C entry point `name` with its device current; raises unless it returns MHC_OK."""
    with torch.cuda.device(device):
        st = getattr(load(), name)(*args)
    if st != MHC_OK:
        raise LayerError(st, name)


def _scratch(nbytes: int, device, stream):
    """A workspace, kept from reuse until the work on a stream of the caller's is done."""
    if not nbytes:
        return None
    t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        t.record_stream(stream)
    return t


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


# ---------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------

def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
             stream=None):
    """(y, total, rstd): total = x + residual (x itself without one), y its RMS
    norm times weight (FP32 [H]), rstd FP32 [T].  x and residual [T,H], bf16 or
    f16, with any row stride."""
    if stream is None:
        out = (_fast or _compiled()).rms_norm(x, weight, residual, eps, -1)
        if out is not None:
            return out[0], out[2], out[3]
    T, H = _two(x, "x")
    dt, dev = _storage(x, "x"), x.device
    xs = _rows(x, "x", x.dtype, x.shape, dev)
    _flat(weight, "weight", torch.float32, (H,), dev)
    rs = H if residual is None else _rows(residual, "residual", x.dtype, x.shape, dev)
    y = torch.empty((T, H), dtype=x.dtype, device=dev)
    total = None if residual is None else torch.empty((T, H), dtype=x.dtype, device=dev)
    rstd = torch.empty(T, dtype=torch.float32, device=dev)
    _call(dev, "mhc_rms_norm_fwd", x.data_ptr(), _ptr(residual), weight.data_ptr(), y.data_ptr(), _ptr(total),
          rstd.data_ptr(), T, H, xs, rs, eps, dt, _stream_handle(stream, dev))
    return y, (x if total is None else total), rstd


def rms_norm_fp8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                 group: int = 0, stream=None):
    """(y8, scale, total, rstd): as rms_norm, with y in E4M3 and FP32 scales,
    one per row (group = 0: [T,1], as linear_fp8 takes them) or per 128
    channels (group = 128: [T,ceil(H/128)], for a product of the caller's with
    scales along K; linear_fp8 takes one a row); y is about y8 * scale."""
    if stream is None and (group == 0 or group == 128):
        out = (_fast or _compiled()).rms_norm(x, weight, residual, eps, group)
        if out is not None:
            return out
    T, H = _two(x, "x")
    dt, dev = _storage(x, "x"), x.device
    xs = _rows(x, "x", x.dtype, x.shape, dev)
    _flat(weight, "weight", torch.float32, (H,), dev)
    rs = H if residual is None else _rows(residual, "residual", x.dtype, x.shape, dev)
    y = torch.empty((T, H), dtype=_E4M3, device=dev)
    scale = torch.empty((T, 1 if group == 0 else -(-H // 128)), dtype=torch.float32, device=dev)
    total = None if residual is None else torch.empty((T, H), dtype=x.dtype, device=dev)
    rstd = torch.empty(T, dtype=torch.float32, device=dev)
    _call(dev, "mhc_rms_norm_fp8_fwd", x.data_ptr(), _ptr(residual), weight.data_ptr(), y.data_ptr(), scale.data_ptr(),
          _ptr(total), rstd.data_ptr(), T, H, xs, rs, eps, group, dt, _stream_handle(stream, dev))
    return y, scale, (x if total is None else total), rstd


def rms_norm_backward(grad_y: torch.Tensor, total: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                      grad_total: torch.Tensor | None = None, stream=None):
    """(grad_x, grad_weight): the gradients from the gradient of y, the
    forward's total and rstd, and optionally the gradient of total itself.
    grad_x is the gradient of x and of the residual; grad_weight is FP32."""
    if stream is None:
        out = (_fast or _compiled()).rms_norm_backward(grad_y, total, weight, rstd, grad_total)
        if out is not None:
            return out
    T, H = _two(total, "total")
    dt, dev = _storage(total, "total"), total.device
    ss = _rows(total, "total", total.dtype, total.shape, dev)
    gs = _rows(grad_y, "grad_y", total.dtype, total.shape, dev)
    _flat(weight, "weight", torch.float32, (H,), dev)
    _flat(rstd, "rstd", torch.float32, (T,), dev)
    if grad_total is not None:
        _flat(grad_total, "grad_total", total.dtype, total.shape, dev)
    lib = load()
    grad_x = torch.empty((T, H), dtype=total.dtype, device=dev)
    grad_w = torch.empty(H, dtype=torch.float32, device=dev)
    need = lib.mhc_rms_norm_bwd_workspace(T, H)
    ws = _scratch(need, dev, stream)
    _call(dev, "mhc_rms_norm_bwd", grad_y.data_ptr(), total.data_ptr(), weight.data_ptr(), rstd.data_ptr(),
          _ptr(grad_total), grad_x.data_ptr(), grad_w.data_ptr(), _ptr(ws), need, T, H, gs, ss, dt,
          _stream_handle(stream, dev))
    return grad_x, grad_w


# ---------------------------------------------------------------------------
# matrix product
# ---------------------------------------------------------------------------

def _activation(name: str) -> int:
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {name!r}")
    return code


def _linear(x, x_scale, w, w_scale, bias, activation, residual, out_dtype, keep, stream):
    T, I = _two(x, "x")
    O, Iw = _two(w, "weight")
    dev = x.device
    fp8 = x_scale is not None
    act = _activation(activation)
    dt = _DTYPES.get(out_dtype)
    if dt is None:
        raise TypeError(f"{'dtype' if fp8 else 'x'} must be bfloat16 or float16, got {out_dtype}")
    operand = _E4M3 if fp8 else out_dtype
    xs = _rows(x, "x", operand, x.shape, dev)
    ws = _rows(w, "weight", operand, (O, I), dev)
    if fp8:
        # one scale per row; rms_norm_fp8's [T,1] is as good as [T]
        _flat(x_scale, "x_scale", torch.float32, (T, 1) if x_scale.dim() == 2 else (T,), dev)
        _flat(w_scale, "w_scale", torch.float32, (O, 1) if w_scale.dim() == 2 else (O,), dev)
    if bias is not None:
        _flat(bias, "bias", torch.float32, (O,), dev)
    rs = O if residual is None else _rows(residual, "residual", out_dtype, (T, O), dev)
    lib = load()
    y = torch.empty((T, O), dtype=out_dtype, device=dev)
    z = torch.empty((T, O), dtype=out_dtype, device=dev) if keep else None
    xp, wp = x.data_ptr(), w.data_ptr()
    need = lib.mhc_linear_workspace(T, I, O, xs, ws, 1 if fp8 else 2, 0 if (xp | wp) & 15 else 1)
    work = _scratch(need, dev, stream)
    sh = _stream_handle(stream, dev)
    if fp8:
        _call(dev, "mhc_linear_fp8_fwd", xp, x_scale.data_ptr(), wp, w_scale.data_ptr(), _ptr(bias), _ptr(residual),
              y.data_ptr(), _ptr(z), _ptr(work), need, T, I, O, xs, ws, rs, act, dt, sh)
    else:
        _call(dev, "mhc_linear_fwd", xp, wp, _ptr(bias), _ptr(residual), y.data_ptr(), _ptr(z), _ptr(work), need, T, I, O,
              xs, ws, rs, act, dt, sh)
    return y, z


def linear(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, activation: str = "none",
           residual: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """act(x weight^T + bias) + residual: x [T,I], weight [O,I], residual and
    the result [T,O], all bf16 or all f16 (x, weight and residual with any row
    stride); bias FP32 [O]; activation "none", "relu", "silu" or "gelu"."""
    if stream is None and activation in ACTIVATIONS:
        out = (_fast or _compiled()).linear(x, None, weight, None, bias, ACTIVATIONS[activation], residual, -1, False)
        if out is not None:
            return out[0]
    return _linear(x, None, weight, None, bias, activation, residual, x.dtype, False, stream)[0]


def linear_preact(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, activation: str = "none",
                  residual: torch.Tensor | None = None, stream=None):
    """(y, z): as linear, and the pre-activation z = x weight^T + bias that linear_backward reads."""
    if stream is None and activation in ACTIVATIONS:
        out = (_fast or _compiled()).linear(x, None, weight, None, bias, ACTIVATIONS[activation], residual, -1, True)
        if out is not None:
            return out
    return _linear(x, None, weight, None, bias, activation, residual, x.dtype, True, stream)


def linear_fp8(x8: torch.Tensor, x_scale: torch.Tensor, w8: torch.Tensor, w_scale: torch.Tensor,
               bias: torch.Tensor | None = None, activation: str = "none", residual: torch.Tensor | None = None,
               dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """The product of E4M3 operands x8 [T,I] and w8 [O,I] with one FP32 scale
    per row of each (x_scale [T] or [T,1], w_scale [O] or [O,1]); residual and
    the result are of `dtype`."""
    if stream is None and activation in ACTIVATIONS and dtype in _DTYPES and x_scale is not None:
        out = (_fast or _compiled()).linear(x8, x_scale, w8, w_scale, bias, ACTIVATIONS[activation], residual,
                                            _DTYPES[dtype], False)
        if out is not None:
            return out[0]
    if not isinstance(x_scale, torch.Tensor) or not isinstance(w_scale, torch.Tensor):
        raise TypeError("x_scale and w_scale must be torch.Tensors")
    return _linear(x8, x_scale, w8, w_scale, bias, activation, residual, dtype, False, stream)[0]


def linear_backward(grad_y: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, z: torch.Tensor | None = None,
                    activation: str = "none", bias: bool = True, want=(True, True), stream=None):
    """(grad_x, grad_weight, grad_bias) of linear, from the gradient of y and,
    with an activation, the forward's z (all of them dense).  grad_bias is FP32,
    None when `bias` is false; `want` says which of grad_x and grad_weight to
    compute.  Both read grad_y * act'(z) rounded to the storage type, as the
    tensor cores take it; grad_bias sums it unrounded."""
    if stream is None and activation in ACTIVATIONS:
        out = (_fast or _compiled()).linear_backward(grad_y, x, weight, z, ACTIVATIONS[activation], bias, want[0], want[1])
        if out is not None:
            return out
    T, I = _two(x, "x")
    O, _ = _two(weight, "weight")
    dt, dev = _storage(x, "x"), x.device
    act = _activation(activation)
    _flat(x, "x", x.dtype, x.shape, dev)
    _flat(weight, "weight", x.dtype, (O, I), dev)
    _flat(grad_y, "grad_y", x.dtype, (T, O), dev)
    if act != 0:
        if z is None:
            raise ValueError("an activation's backward needs z")
        _flat(z, "z", x.dtype, (T, O), dev)
    lib = load()
    grad_x = torch.empty((T, I), dtype=x.dtype, device=dev) if want[0] else None
    grad_w = torch.empty((O, I), dtype=x.dtype, device=dev) if want[1] else None
    grad_b = torch.empty(O, dtype=torch.float32, device=dev) if bias else None
    gp, xp, wp = grad_y.data_ptr(), x.data_ptr(), weight.data_ptr()
    need = lib.mhc_linear_bwd_workspace(T, I, O, act, int(want[0]), int(want[1]), int(bias),
                                        0 if (gp | xp | wp) & 15 else 1)
    work = _scratch(need, dev, stream)
    _call(dev, "mhc_linear_bwd", gp, xp, wp, _ptr(z if act else None), _ptr(grad_x), _ptr(grad_w), _ptr(grad_b),
          _ptr(work), need, T, I, O, act, dt, _stream_handle(stream, dev))
    return grad_x, grad_w, grad_b


# ---------------------------------------------------------------------------
# gated product
# ---------------------------------------------------------------------------

def _gated(x, x_scale, w, w_scale, bias, activation, out_dtype, keep, stream):
    T, I = _two(x, "x")
    O, _ = _two(w, "weight")
    dev = x.device
    fp8 = x_scale is not None
    act = _activation(activation)
    dt = _DTYPES.get(out_dtype)
    if dt is None:
        raise TypeError(f"{'dtype' if fp8 else 'x'} must be bfloat16 or float16, got {out_dtype}")
    if O % 2:
        raise ValueError(f"weight must have the gate's and as many of the up projection's rows, got {tuple(w.shape)}")
    operand = _E4M3 if fp8 else out_dtype
    xs = _rows(x, "x", operand, x.shape, dev)
    ws = _rows(w, "weight", operand, (O, I), dev)
    if fp8:
        _flat(x_scale, "x_scale", torch.float32, (T, 1) if x_scale.dim() == 2 else (T,), dev)
        _flat(w_scale, "w_scale", torch.float32, (O, 1) if w_scale.dim() == 2 else (O,), dev)
    if bias is not None:
        _flat(bias, "bias", torch.float32, (O,), dev)
    lib = load()
    y = torch.empty((T, O // 2), dtype=out_dtype, device=dev)
    z = torch.empty((T, O), dtype=out_dtype, device=dev) if keep else None
    xp, wp = x.data_ptr(), w.data_ptr()
    need = lib.mhc_linear_workspace(T, I, O, xs, ws, 1 if fp8 else 2, 0 if (xp | wp) & 15 else 1)
    work = _scratch(need, dev, stream)
    sh = _stream_handle(stream, dev)
    if fp8:
        _call(dev, "mhc_gated_linear_fp8_fwd", xp, x_scale.data_ptr(), wp, w_scale.data_ptr(), _ptr(bias), y.data_ptr(),
              _ptr(z), _ptr(work), need, T, I, O // 2, xs, ws, act, dt, sh)
    else:
        _call(dev, "mhc_gated_linear_fwd", xp, wp, _ptr(bias), y.data_ptr(), _ptr(z), _ptr(work), need, T, I, O // 2, xs, ws,
              act, dt, sh)
    return y, z


def gated_linear(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, activation: str = "silu",
                 stream=None) -> torch.Tensor:
    """act(x w_gate^T + b_gate) * (x w_up^T + b_up), the first half of a gated
    feed-forward, in one kernel: x [T,I], weight [2F,I] (the gate's F rows,
    then the up projection's), the result [T,F], all bf16 or all f16 (x and
    weight with any row stride); bias FP32 [2F]; activation as in `linear`."""
    if stream is None and activation in ACTIVATIONS:
        out = (_fast or _compiled()).gated_linear(x, None, weight, None, bias, ACTIVATIONS[activation], -1, False)
        if out is not None:
            return out[0]
    return _gated(x, None, weight, None, bias, activation, x.dtype if isinstance(x, torch.Tensor) else None, False, stream)[0]


def gated_linear_preact(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, activation: str = "silu",
                        stream=None):
    """(y, z): as gated_linear, and z = x weight^T + bias [T,2F] that gated_linear_backward reads."""
    if stream is None and activation in ACTIVATIONS:
        out = (_fast or _compiled()).gated_linear(x, None, weight, None, bias, ACTIVATIONS[activation], -1, True)
        if out is not None:
            return out
    return _gated(x, None, weight, None, bias, activation, x.dtype if isinstance(x, torch.Tensor) else None, True, stream)


def gated_linear_fp8(x8: torch.Tensor, x_scale: torch.Tensor, w8: torch.Tensor, w_scale: torch.Tensor,
                     bias: torch.Tensor | None = None, activation: str = "silu", dtype: torch.dtype = torch.bfloat16,
                     stream=None) -> torch.Tensor:
    """gated_linear of E4M3 operands x8 [T,I] and w8 [2F,I] with one FP32 scale
    per row of each (x_scale [T] or [T,1], w_scale [2F] or [2F,1]); the result
    is of `dtype`."""
    if stream is None and activation in ACTIVATIONS and dtype in _DTYPES and x_scale is not None:
        out = (_fast or _compiled()).gated_linear(x8, x_scale, w8, w_scale, bias, ACTIVATIONS[activation], _DTYPES[dtype],
                                                  False)
        if out is not None:
            return out[0]
    if not isinstance(x_scale, torch.Tensor) or not isinstance(w_scale, torch.Tensor):
        raise TypeError("x_scale and w_scale must be torch.Tensors")
    return _gated(x8, x_scale, w8, w_scale, bias, activation, dtype, False, stream)[0]


def gated_linear_backward(grad_y: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, z: torch.Tensor,
                          activation: str = "silu", bias: bool = True, want=(True, True), stream=None):
    """(grad_x, grad_weight, grad_bias) of gated_linear, from the gradient of y
    and the forward's z (both dense; x and weight with any row stride).
    grad_bias is FP32 [2F], None when `bias` is false; `want` says which of
    grad_x and grad_weight to compute.  Both read the gradient of z rounded to
    the storage type, as the tensor cores take it; grad_bias sums it unrounded."""
    if stream is None and activation in ACTIVATIONS:
        out = (_fast or _compiled()).gated_linear_backward(grad_y, x, weight, z, ACTIVATIONS[activation], bias, want[0],
                                                           want[1])
        if out is not None:
            return out
    T, I = _two(x, "x")
    O, _ = _two(weight, "weight")
    dt, dev = _storage(x, "x"), x.device
    act = _activation(activation)
    if O % 2:
        raise ValueError(f"weight must have the gate's and as many of the up projection's rows, got {tuple(weight.shape)}")
    xs = _rows(x, "x", x.dtype, x.shape, dev)
    ws = _rows(weight, "weight", x.dtype, (O, I), dev)
    _flat(grad_y, "grad_y", x.dtype, (T, O // 2), dev)
    _flat(z, "z", x.dtype, (T, O), dev)
    lib = load()
    grad_x = torch.empty((T, I), dtype=x.dtype, device=dev) if want[0] else None
    grad_w = torch.empty((O, I), dtype=x.dtype, device=dev) if want[1] else None
    grad_b = torch.empty(O, dtype=torch.float32, device=dev) if bias else None
    xp, wp = x.data_ptr(), weight.data_ptr()
    need = lib.mhc_gated_linear_bwd_workspace(T, I, O // 2, xs, ws, int(want[0]), int(want[1]), int(bias),
                                              0 if (xp | wp) & 15 else 1)
    work = _scratch(need, dev, stream)
    _call(dev, "mhc_gated_linear_bwd", grad_y.data_ptr(), xp, wp, z.data_ptr(), _ptr(grad_x), _ptr(grad_w), _ptr(grad_b),
          _ptr(work), need, T, I, O // 2, xs, ws, act, dt, _stream_handle(stream, dev))
    return grad_x, grad_w, grad_b


# ---------------------------------------------------------------------------
# cross entropy over a vocabulary
# ---------------------------------------------------------------------------

def linear_cross_entropy(x: torch.Tensor, weight: torch.Tensor, target: torch.Tensor, stream=None):
    """(loss, lse), FP32 [T], of the logits x weight^T, which are not kept (sums
    of a small vocabulary's pass through the workspace): lse their logsumexp,
    loss = lse - logit of the target.  x [T,I] and weight [V,I], both bf16 or
    both f16, with any row stride; target int64 [T].  A token whose target is
    outside 0 .. V-1 (-100, by custom) is ignored: loss 0.  The mean over the
    others is the caller's division by their number."""
    if stream is None:
        out = (_fast or _compiled()).linear_cross_entropy(x, weight, target)
        if out is not None:
            return out
    T, I = _two(x, "x")
    V, _ = _two(weight, "weight")
    dt, dev = _storage(x, "x"), x.device
    xs = _rows(x, "x", x.dtype, x.shape, dev)
    ws = _rows(weight, "weight", x.dtype, (V, I), dev)
    _flat(target, "target", torch.int64, (T,), dev)
    lib = load()
    loss, lse = (torch.empty(T, dtype=torch.float32, device=dev) for _ in range(2))
    xp, wp = x.data_ptr(), weight.data_ptr()
    need = lib.mhc_linear_cross_entropy_workspace(T, I, V, xs, ws, 0 if (xp | wp) & 15 else 1)
    work = _scratch(need, dev, stream)
    _call(dev, "mhc_linear_cross_entropy_fwd", xp, wp, target.data_ptr(), loss.data_ptr(), lse.data_ptr(), _ptr(work), need,
          T, I, V, xs, ws, dt, _stream_handle(stream, dev))
    return loss, lse


def linear_cross_entropy_backward(grad_loss: torch.Tensor | None, x: torch.Tensor, weight: torch.Tensor,
                                  target: torch.Tensor, lse: torch.Tensor, grad_lse: torch.Tensor | None = None,
                                  want=(True, True), stream=None):
    """(grad_x, grad_weight) of linear_cross_entropy, from the gradients of loss
    and lse (FP32 [T]; either may be None) and the forward's lse; `want` says
    which of the two to compute.  The logits are computed again and their
    gradient is in the workspace by pieces of the vocabulary (whole up to 2^27
    values, 256 MB); both products read their gradient rounded to the storage
    type (after a scaling, so that f16 holds small probabilities and a gradient
    that all tokens share, as that of a mean, is not rounded)."""
    if stream is None:
        out = (_fast or _compiled()).linear_cross_entropy_backward(grad_loss, x, weight, target, lse, grad_lse, want[0],
                                                                   want[1])
        if out is not None:
            return out
    T, I = _two(x, "x")
    V, _ = _two(weight, "weight")
    dt, dev = _storage(x, "x"), x.device
    xs = _rows(x, "x", x.dtype, x.shape, dev)
    ws = _rows(weight, "weight", x.dtype, (V, I), dev)
    _flat(target, "target", torch.int64, (T,), dev)
    _flat(lse, "lse", torch.float32, (T,), dev)
    if grad_loss is None and grad_lse is None:
        raise ValueError("one of grad_loss and grad_lse must be given")
    for t, name in ((grad_loss, "grad_loss"), (grad_lse, "grad_lse")):
        if t is not None:
            _flat(t, name, torch.float32, (T,), dev)
    lib = load()
    grad_x = torch.empty((T, I), dtype=x.dtype, device=dev) if want[0] else None
    grad_w = torch.empty((V, I), dtype=x.dtype, device=dev) if want[1] else None
    xp, wp = x.data_ptr(), weight.data_ptr()
    need = lib.mhc_linear_cross_entropy_bwd_workspace(T, I, V, xs, ws, int(want[0]), int(want[1]), 0 if (xp | wp) & 15 else 1)
    work = _scratch(need, dev, stream)
    _call(dev, "mhc_linear_cross_entropy_bwd", _ptr(grad_loss), _ptr(grad_lse), xp, wp, target.data_ptr(), lse.data_ptr(),
          _ptr(grad_x), _ptr(grad_w), _ptr(work), need, T, I, V, xs, ws, dt, _stream_handle(stream, dev))
    return grad_x, grad_w


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

def rotary_frequencies(dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                       trained: int = 4096, fast: float = 32.0, slow: float = 1.0, device="cuda") -> torch.Tensor:
    """The FP32 table [dim/2] of a head's rotated part of `dim` values:
    f_j = base^(-2j/dim), with `scaling` for contexts `factor` times the
    trained length: "linear" divides every frequency by the factor; "ntk"
    raises the base so that the slowest one is divided by it; "yarn" (Peng et
    al., 2023, "NTK-by-parts") goes by the turns r_j = trained f_j / (2 pi) that
    a pair makes over the trained length: f_j (k + (1 - k) / factor), where
    k = (r_j - slow) / (fast - slow), held within 0 and 1.  That ramp is linear
    in the turns.  Checkpoints whose table ramps linearly in the channel index
    j between the two bounds differ in the channels between; their table goes
    to `rotary` as it is, like any other.  The magnitude that goes with a
    scaling (0.1 ln(factor) + 1 for "yarn") is `rotary`'s scale."""
    if dim <= 0 or dim % 2:
        raise ValueError(f"dim must be positive and even, got {dim}")
    if scaling == "ntk" and dim > 2:
        base = base * factor ** (dim / (dim - 2))
    f = float(base) ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        turns = trained * f / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"scaling must be none, linear, ntk or yarn, got {scaling!r}")
    return f.float().to(device)


def rotary(x: torch.Tensor, positions: torch.Tensor, frequencies: torch.Tensor, interleaved: bool = False,
           scale: float = 1.0, inverse: bool = False, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x [T,heads,D] (bf16 or f16) with the first R = 2 len(frequencies) values
    of each head rotated by positions[t] * frequencies[j] and multiplied by
    `scale`; pairs are (j, j + R/2), or (2j, 2j + 1) when interleaved.  x's
    heads are contiguous and lie in either order, tokens or heads outermost,
    with any distances at which they do not overlap.  positions int64 [T].
    inverse rotates back (the gradient).  `out`, tokens outermost, may be x
    itself."""
    if stream is None and out is None:
        done = (_fast or _compiled()).rotary(x, positions, frequencies, interleaved, float(scale), inverse)
        if done is not None:
            return done[0]
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.dim() != 3:
        raise ValueError(f"x must be [T,heads,D], got {tuple(x.shape)}")
    T, heads, D = x.shape
    dt, dev = _storage(x, "x"), x.device
    if dev.type != "cuda":
        raise ValueError(f"x must be a CUDA tensor, got {dev}")
    _flat(positions, "positions", torch.int64, (T,), dev)
    _flat(frequencies, "frequencies", torch.float32, frequencies.shape, dev)
    if frequencies.dim() != 1:
        raise ValueError("frequencies must be 1-d")
    if out is None:
        out = torch.empty((T, heads, D), dtype=x.dtype, device=dev)
    elif out.shape != x.shape or out.dtype != x.dtype or out.device != dev:
        raise ValueError(f"out must be {x.dtype} {tuple(x.shape)} on {dev}")
    strides = []
    for t, name in ((x, "x"), (out, "out")):
        token, head, one = t.stride()
        if one != 1 and D > 1:
            raise ValueError(f"{name}'s heads must be contiguous, got strides {t.stride()}")
        head = head if heads > 1 else D
        row = max(heads - 1, 0) * head + D
        token = token if T > 1 else row
        if name == "x" and T > 0 and heads > 0 and (head < D or token < D or (token < row and head < (T - 1) * token + D)):
            raise ValueError(f"x's heads must not overlap, got strides {t.stride()}")
        strides += [token, head]
    _call(dev, "mhc_rotary", x.data_ptr(), positions.data_ptr(), frequencies.data_ptr(), out.data_ptr(), T, heads, D,
          2 * frequencies.shape[0], *strides, scale, int(interleaved), int(inverse), dt, _stream_handle(stream, dev))
    return out
