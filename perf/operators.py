"""The layer operators' cases: RMS norm (with the residual's addition, an 8-bit output and its
gradient), matrix product (with bias, activation and residual, 8-bit operands and its gradients),
and rotary positions.  Each case has a plain form in 32-bit torch operations and the framework's
own call.

``own`` selects which of the two ``run`` computes; both read the same ``prepare`` state.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -60


def listed():
    return [
        # one decoded token between two sublayers: the sum, its norm and the next product's 8-bit operand
        dict(name="norm_decode_fp8", op="norm", out="fp8", T=1, H=7168, group=0, residual=True, dtype="bf16"),
        # a 4096-token training or prefill pass at the model's width
        dict(name="norm_prefill", op="norm", out="same", T=4096, H=7168, group=0, residual=True, dtype="bf16"),
        # the longest prefill, 8-bit output with a scale per 128 channels
        dict(name="norm_long_fp8", op="norm", out="fp8", T=65536, H=7168, group=128, residual=True, dtype="bf16"),
        # the training pass's gradients
        dict(name="norm_bwd", op="norm_bwd", T=4096, H=7168, residual=True, dtype="bf16"),
        # odd rows, no two of them at the same alignment
        dict(name="norm_bwd_odd", op="norm_bwd", T=3001, H=1279, residual=False, dtype="f16"),
        # one decoded token through a square product
        dict(name="linear_decode", op="linear", T=1, I=7168, O=7168, activation="silu", bias=True, residual=False,
             dtype="bf16"),
        # a batch of decoded tokens through an 8-bit up projection
        dict(name="linear_decode_fp8", op="linear_fp8", T=64, I=7168, O=14336, activation="none", bias=False,
             residual=True, dtype="bf16"),
        # a prefill or training forward pass
        dict(name="linear_prefill", op="linear", T=4096, I=7168, O=7168, activation="gelu", bias=True, residual=True,
             dtype="bf16"),
        # odd sizes everywhere
        dict(name="linear_odd", op="linear", T=129, I=1279, O=4097, activation="silu", bias=True, residual=True,
             dtype="f16"),
        # the training pass's gradients
        dict(name="linear_bwd", op="linear_bwd", T=4096, I=4096, O=7168, activation="silu", bias=True, dtype="bf16"),
        # one new token of each of 128 requests, at its own position
        dict(name="rotary_decode", op="rotary", T=128, heads=40, other=8, D=128, R=128, interleaved=False,
             inverse=False, longest=131072, stretch=4.0, dtype="bf16"),
        # a long prefill, the first half of each head rotated, in the interleaved layout
        dict(name="rotary_prefill", op="rotary", T=32768, heads=40, other=8, D=128, R=64, interleaved=True,
             inverse=False, longest=32768, stretch=1.0, dtype="f16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A row length: mostly of whole 16-byte vectors, at times odd."""
    n = _log_int(rng, lo, hi)
    return n // 8 * 8 if rng.random() < 0.7 else n


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "linear", "linear", "linear_fp8", "linear_bwd", "rotary"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op in ("norm", "norm_bwd"):
        H = _width(rng, 256, 8192)
        case = dict(op=op, T=_log_int(rng, 1, min(65536, 65536 * 7168 // H)), H=H, residual=rng.random() < 0.7,
                    dtype=dtype)
        if op == "norm":
            case["out"] = rng.choice(["same", "fp8"])
            case["group"] = rng.choice([0, 128]) if case["out"] == "fp8" else 0
        else:
            case["T"] = min(case["T"], max(1, 4096 * 7168 * 8 // H))
        return case
    if op in ("linear", "linear_fp8", "linear_bwd"):
        I = _width(rng, 256, 8192)
        O = _width(rng, 24, 16384)
        most = 4096 * 7168 * 7168 // (I * O)
        if op == "linear_bwd":
            most = most // 2
        case = dict(op=op, T=_log_int(rng, 1, max(1, min(16384, most))), I=I, O=O,
                    activation=rng.choice(["none", "relu", "silu", "gelu"]), bias=rng.random() < 0.6, dtype=dtype)
        if op == "linear_fp8":
            case["I"] = max(16, I // 16 * 16)
        if op != "linear_bwd":
            case["residual"] = rng.random() < 0.5
        return case
    D = rng.choice([64, 80, 96, 128, 192, 256])
    heads = rng.choice([1, 5, 8, 16, 40, 64])
    return dict(op="rotary", T=_log_int(rng, 1, 32768 * 40 * 128 // (heads * D)), heads=heads, other=rng.choice([0, 1, 8]),
                D=D, R=rng.choice([D, D // 2, D // 4]), interleaved=rng.random() < 0.5, inverse=rng.random() < 0.4,
                longest=_log_int(rng, 2048, 131072), stretch=rng.choice([1.0, 4.0, 8.0]), dtype=dtype)


def _frequencies(R, stretch):
    """Base 10000, the slow half of the spectrum slowed down by `stretch`."""
    f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    return torch.where(f < f[f.numel() // 2], f / stretch, f).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, spread=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * spread

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    op, dt = case["op"], DTYPES[case["dtype"]]
    s = dict(case)
    if op in ("norm", "norm_bwd"):
        T, H = case["T"], case["H"]
        # tokens of different magnitude, a few channels that stand out
        level = torch.exp2(3 * uniform(T, 1) - 1) * (1 + 15 * (uniform(1, H) > 0.995))
        s["x"] = (normal(T, H) * level).to(dt)
        s["r"] = (normal(T, H) * level).to(dt) if case["residual"] else None
        s["w"] = 1 + normal(H, spread=0.2)
        s["eps"] = 1e-6
        if op == "norm_bwd":
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(-1) + s["eps"])
            s["g"] = normal(T, H).to(dt)
    elif op == "rotary":
        T, n, D = case["T"], case["heads"], case["D"]
        # the rotated heads are the first of each row of a larger product's output
        rows = normal(T, (n + case["other"]) * D).to(dt)
        s["x"] = rows[:, :n * D].view(T, n, D)
        s["pos"] = torch.randint(0, case["longest"], (T,), generator=gen, device="cuda", dtype=torch.int64)
        s["f"] = _frequencies(case["R"], case["stretch"]).cuda()
        s["scale"] = 1.0 + 0.1 * math.log(case["stretch"])
    else:
        T, I, O = case["T"], case["I"], case["O"]
        x, w = normal(T, I), normal(O, I, spread=I ** -0.5)
        if op == "linear_fp8":
            s["sx"] = x.abs().amax(-1) / E4M3_MAX
            s["sw"] = w.abs().amax(-1) / E4M3_MAX
            s["x"] = (x / s["sx"][:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            s["w"] = (w / s["sw"][:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        else:
            s["x"], s["w"] = x.to(dt), w.to(dt)
        s["b"] = normal(O, spread=0.5) if case["bias"] else None
        if op == "linear_bwd":
            s["z"] = normal(T, O).to(dt) if case["activation"] != "none" else None
            s["g"] = normal(T, O).to(dt)
        else:
            s["r"] = normal(T, O).to(dt) if case["residual"] else None
    return s


# ---------------------------------------------------------------------------
# plain forms: 32-bit torch operations, one rounding at the end
# ---------------------------------------------------------------------------

def _activation(z, kind):
    if kind == "relu":
        return z * (z > 0)
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    if kind == "gelu":
        return z * 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _slope(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    return torch.ones_like(z)


def _groups(y, group):
    """`y` as [T, groups, group], zeros past its end."""
    T, H = y.shape
    size = group or H
    n = -(-H // size)
    padded = torch.zeros(T, n * size, dtype=y.dtype, device=y.device)
    padded[:, :H] = y
    return padded.view(T, n, size)


def _plain_norm(s):
    dt = DTYPES[s["dtype"]]
    total = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
    rstd = 1 / torch.sqrt((total * total).sum(-1) / s["H"] + s["eps"])
    y = total * rstd[:, None] * s["w"]
    out = {"rstd": rstd}
    if s["r"] is not None:
        out["total"] = total.to(dt)
    if s["out"] == "same":
        out["y"] = y.to(dt)
        return out
    parts = _groups(y, s["group"])
    amax = parts.abs().amax(-1).clamp(min=AMAX_FLOOR)
    q = (parts * (E4M3_MAX / amax)[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    out["y"] = q.view(s["T"], -1)[:, :s["H"]].to(torch.float8_e4m3fn)
    out["scale"] = amax / E4M3_MAX
    return out


def _plain_norm_bwd(s):
    dt = DTYPES[s["dtype"]]
    xhat = s["x"].float() * s["rstd"][:, None]
    g = s["g"].float()
    gw = g * s["w"]
    grad = s["rstd"][:, None] * (gw - xhat * ((gw * xhat).sum(-1, keepdim=True) / s["H"]))
    if s["r"] is not None:
        grad = grad + s["r"].float()          # the gradient that reaches the sum past the norm
    return {"grad_x": grad.to(dt), "grad_w": (g * xhat).sum(0)}


def _plain_linear(s):
    dt = DTYPES[s["dtype"]]
    z = s["x"].float() @ s["w"].float().t()
    if s["op"] == "linear_fp8":
        z = z * s["sx"][:, None] * s["sw"]
    if s["b"] is not None:
        z = z + s["b"]
    y = _activation(z, s["activation"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return {"y": y.to(dt)}


def _plain_linear_bwd(s):
    dt = DTYPES[s["dtype"]]
    g = s["g"].float()
    if s["activation"] != "none":
        g = g * _slope(s["z"].float(), s["activation"])
    out = {"grad_x": (g @ s["w"].float()).to(dt), "grad_w": (g.t() @ s["x"].float()).to(dt)}
    if s["b"] is not None:
        out["grad_b"] = g.sum(0)
    return out


def _plain_rotary(s):
    x, R = s["x"].float(), s["R"]
    angle = s["pos"].float()[:, None] * s["f"]
    cos, sin = (torch.cos(angle) * s["scale"])[:, None], (torch.sin(angle) * s["scale"])[:, None]
    if s["inverse"]:
        sin = -sin
    y = x.clone()
    if s["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2], y[..., 1:R:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y[..., :R // 2], y[..., R // 2:R] = a * cos - b * sin, b * cos + a * sin
    return {"y": y.to(DTYPES[s["dtype"]])}


_PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "linear": _plain_linear, "linear_fp8": _plain_linear,
          "linear_bwd": _plain_linear_bwd, "rotary": _plain_rotary}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own(s):
    from invariant_mhc_aggregate_gb300 import layer
    op = s["op"]
    if op == "norm":
        if s["out"] == "same":
            y, total, rstd = layer.rms_norm(s["x"], s["w"], residual=s["r"], eps=s["eps"])
            out = {"y": y, "rstd": rstd}
        else:
            y, scale, total, rstd = layer.rms_norm_fp8(s["x"], s["w"], residual=s["r"], eps=s["eps"], group=s["group"])
            out = {"y": y, "rstd": rstd, "scale": scale}
        if s["r"] is not None:
            out["total"] = total
        return out
    if op == "norm_bwd":
        grad_x, grad_w = layer.rms_norm_backward(s["g"], s["x"], s["w"], s["rstd"], grad_total=s["r"])
        return {"grad_x": grad_x, "grad_w": grad_w}
    if op == "linear":
        return {"y": layer.linear(s["x"], s["w"], bias=s["b"], activation=s["activation"], residual=s["r"])}
    if op == "linear_fp8":
        return {"y": layer.linear_fp8(s["x"], s["sx"], s["w"], s["sw"], bias=s["b"], activation=s["activation"],
                                      residual=s["r"], dtype=DTYPES[s["dtype"]])}
    if op == "linear_bwd":
        grad_x, grad_w, grad_b = layer.linear_backward(s["g"], s["x"], s["w"], z=s["z"], activation=s["activation"],
                                                       bias=s["b"] is not None)
        out = {"grad_x": grad_x, "grad_w": grad_w}
        if grad_b is not None:
            out["grad_b"] = grad_b
        return out
    return {"y": layer.rotary(s["x"], s["pos"], s["f"], interleaved=s["interleaved"], scale=s["scale"],
                              inverse=s["inverse"])}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


def work(case):
    op, T = case["op"], case["T"]
    if op in ("norm", "norm_bwd"):
        H = case["H"]
        if op == "norm":
            size = 1 if case["out"] == "fp8" else 2
            scales = T * (-(-H // (case["group"] or H))) * 4 if case["out"] == "fp8" else 0
            return {"bytes": T * H * (2 + (4 if case["residual"] else 0) + size) + 4 * H + 4 * T + scales,
                    "flops": 5 * T * H}
        return {"bytes": T * H * (6 + (2 if case["residual"] else 0)) + 8 * H + 4 * T, "flops": 10 * T * H}
    if op == "rotary":
        return {"bytes": 4 * T * case["heads"] * case["D"] + 8 * T + 2 * case["R"],
                "flops": 3 * T * case["heads"] * case["R"]}
    I, O = case["I"], case["O"]
    if op == "linear_bwd":
        z = T * O if case["activation"] != "none" else 0
        return {"bytes": 2 * (T * O + z + 2 * T * I + 2 * O * I) + (4 * O if case["bias"] else 0), "flops": 4 * T * I * O}
    size = 1 if op == "linear_fp8" else 2
    return {"bytes": size * (T * I + O * I) + 2 * T * O * (2 if case["residual"] else 1) + (4 * O if case["bias"] else 0)
            + (4 * (T + O) if op == "linear_fp8" else 0), "flops": 2 * T * I * O}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _slope64(z, kind):
    """The activation's derivative by its own formula, value by value."""
    if kind == "relu":
        return torch.where(z > 0, 1.0, 0.0).double()
    if kind == "silu":
        p = torch.special.expit(z)
        return p + z * p * (1 - p)
    return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    wide = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    x = wide["x"]
    if op == "norm":
        v = x if wide["r"] is None else x.add_(wide["r"])
        rms = torch.linalg.vector_norm(v, dim=-1).square().div(case["H"]).add(s["eps"]).sqrt()
        y = v / rms[:, None]
        y *= wide["w"]
        out = {"rstd": rms.reciprocal()}
        if wide["r"] is not None:
            out["total"] = v
        if case["out"] == "same":
            out["y"] = y
            return out
        size = case["group"] or case["H"]
        scale = torch.stack([p.abs().amax(-1) for p in y.split(size, dim=-1)], -1).clamp(min=AMAX_FLOOR) / E4M3_MAX
        out["scale"] = scale
        out["y"] = y / scale.repeat_interleave(size, dim=-1)[:, :case["H"]]
        return out
    if op == "norm_bwd":
        r = wide["rstd"][:, None]
        gw = wide["g"] * wide["w"]
        grad = r * gw - x * r ** 3 * torch.einsum("th,th->t", gw, x)[:, None] / case["H"]
        return {"grad_x": grad if wide["r"] is None else grad + wide["r"],
                "grad_w": torch.einsum("th,th,t->h", wide["g"], x, wide["rstd"])}
    if op == "rotary":
        turn = wide["pos"][:, None] * wide["f"]
        phase = torch.polar(torch.full_like(turn, s["scale"]), -turn if case["inverse"] else turn)[:, None]
        R, y = case["R"], x.clone()
        if case["interleaved"]:
            y[..., :R] = torch.view_as_real(torch.complex(x[..., 0:R:2], x[..., 1:R:2]) * phase).flatten(-2)
        else:
            v = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * phase
            y[..., :R] = torch.cat([v.real, v.imag], -1)
        return {"y": y}
    if op == "linear_bwd":
        g = wide["g"]
        if case["activation"] != "none":
            g = g * _slope64(wide["z"], case["activation"])
        out = {"grad_x": torch.einsum("to,oi->ti", g, wide["w"]), "grad_w": torch.einsum("to,ti->oi", g, x)}
        if wide["b"] is not None:
            out["grad_b"] = torch.einsum("to->o", g)
        return out
    if op == "linear_fp8":
        x, wide["w"] = x * wide["sx"][:, None], wide["w"] * wide["sw"][:, None]
    z = torch.einsum("ti,oi->to", x, wide["w"])
    if wide["b"] is not None:
        z = z + wide["b"]
    if case["activation"] == "relu":
        z = z.clamp(min=0)
    elif case["activation"] == "silu":
        z = z * torch.special.expit(z)
    elif case["activation"] == "gelu":
        z = z * torch.special.ndtr(z)
    return {"y": z if wide["r"] is None else z + wide["r"]}
