"""The cases of the layer's products that end in more than an epilogue of their own: the gated
product (both projections of a gated feed-forward, the activation and their product; 8-bit
operands; its gradients) and the cross entropy of a product over a large vocabulary (its logits
are not kept; its gradients).  Each case has a plain form in 32-bit torch operations and the
framework's own call.

``own`` selects which of the two ``run`` computes; both read the same ``prepare`` state.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3_MAX = 448.0
IGNORED = -100


def listed():
    return [
        # one decoded token through a feed-forward's gate and up projections
        dict(name="gated_decode", op="gated", T=1, I=2048, F=8192, activation="silu", bias=False, keep=False, dtype="bf16"),
        # a batch of decoded tokens through 8-bit projections
        dict(name="gated_decode_fp8", op="gated_fp8", T=64, I=7168, F=14336, activation="silu", bias=False, keep=False,
             dtype="bf16"),
        # a prefill pass at the model's width
        dict(name="gated_prefill", op="gated", T=4096, I=7168, F=14336, activation="silu", bias=False, keep=False,
             dtype="bf16"),
        # a training forward pass, which keeps what the gradients read
        dict(name="gated_train", op="gated", T=4096, I=4096, F=7168, activation="silu", bias=False, keep=True, dtype="bf16"),
        # odd sizes everywhere
        dict(name="gated_odd", op="gated", T=129, I=1279, F=2731, activation="gelu", bias=True, keep=True, dtype="f16"),
        # the training pass's gradients
        dict(name="gated_bwd", op="gated_bwd", T=4096, I=4096, F=7168, activation="silu", bias=False, dtype="bf16"),
        # the gradients at odd sizes, with a bias
        dict(name="gated_bwd_odd", op="gated_bwd", T=1001, I=1279, F=1365, activation="gelu", bias=True, dtype="f16"),
        # a few tokens scored against a vocabulary: the weight's bytes
        dict(name="ce_few", op="ce", T=8, I=2048, V=32768, ignored=0.0, dtype="bf16"),
        # the loss of a training step
        dict(name="ce_train", op="ce", T=4096, I=7168, V=65536, ignored=0.1, dtype="bf16"),
        # odd sizes everywhere, prompts' tokens ignored
        dict(name="ce_odd", op="ce", T=1023, I=1279, V=50259, ignored=0.4, dtype="f16"),
        # the training step's gradients, with a term that keeps the logsumexp small
        dict(name="ce_bwd", op="ce_bwd", T=4096, I=4096, V=65536, ignored=0.1, spread=True, dtype="bf16"),
        # the gradients at odd sizes, most tokens ignored
        dict(name="ce_bwd_odd", op="ce_bwd", T=513, I=1279, V=32003, ignored=0.7, spread=False, dtype="f16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A row length: mostly of whole 16-byte vectors, at times odd."""
    n = _log_int(rng, lo, hi)
    return n // 8 * 8 if rng.random() < 0.7 else n


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_fp8", "gated_bwd", "ce", "ce", "ce_bwd", "ce_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    I = _width(rng, 256, 8192)
    if op.startswith("gated"):
        F = _width(rng, 24, 16384)
        most = 4096 * 7168 * 14336 // (I * F)
        if op == "gated_bwd":
            most = most // 2
        case = dict(op=op, T=_log_int(rng, 1, max(1, min(16384, most))), I=I, F=F,
                    activation=rng.choice(["silu", "silu", "gelu", "relu", "none"]), bias=rng.random() < 0.4, dtype=dtype)
        if op == "gated_fp8":
            case["I"] = max(16, I // 16 * 16)
        if op != "gated_bwd":
            case["keep"] = op == "gated" and rng.random() < 0.5
        return case
    V = _width(rng, 1000, 131072)
    most = 4096 * 4096 * 65536 // (I * V)
    case = dict(op=op, T=_log_int(rng, 1, max(1, min(8192, most))), I=I, V=V, ignored=rng.choice([0.0, 0.1, 0.5]),
                dtype=dtype)
    if op == "ce_bwd":
        case["spread"] = rng.random() < 0.5
    return case


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, spread=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(spread)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    op, dt = case["op"], DTYPES[case["dtype"]]
    s = dict(case)
    T, I = case["T"], case["I"]
    x = normal(T, I)
    if op.startswith("gated"):
        F = case["F"]
        w = normal(2 * F, I, spread=I ** -0.5)               # the gate's rows, then the up projection's
        if op == "gated_fp8":
            s["sx"] = x.abs().amax(-1) / E4M3_MAX
            s["sw"] = w.abs().amax(-1) / E4M3_MAX
            s["x"] = (x / s["sx"][:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            s["w"] = (w / s["sw"][:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        else:
            s["x"], s["w"] = x.to(dt), w.to(dt)
        s["b"] = normal(2 * F, spread=0.5) if case["bias"] else None
        if op == "gated_bwd":
            s["z"] = normal(T, 2 * F).to(dt)
            s["g"] = normal(T, F).to(dt)
        return s
    V = case["V"]
    w = normal(V, I, spread=2 * I ** -0.5)                   # logits of spread 2
    target = torch.randint(0, V, (T,), generator=gen, device="cuda")
    # a model that has learned: most targets stand out, by up to 14
    x += 14 * uniform(T, 1) * w[target] / 4
    s["x"], s["w"] = x.to(dt), w.to(dt)
    s["target"] = torch.where(uniform(T) < case["ignored"], torch.full_like(target, IGNORED), target)
    if op == "ce_bwd":
        s["lse"] = torch.logsumexp(s["x"].float() @ s["w"].float().t(), -1)
        # of the mean over the tokens that count; binary16 with a loss scale
        count = int((s["target"] >= 0).sum())
        s["g"] = torch.full((T,), (1.0 if dt == torch.bfloat16 else 8192.0) / max(1, count), device="cuda")
        s["g_lse"] = 2e-4 * s["lse"] * s["g"] if case["spread"] else None
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


def _plain_gated(s):
    dt, F = DTYPES[s["dtype"]], s["F"]
    z = s["x"].float() @ s["w"].float().t()
    if s["op"] == "gated_fp8":
        z = z * s["sx"][:, None] * s["sw"]
    if s["b"] is not None:
        z = z + s["b"]
    out = {"y": (_activation(z[:, :F], s["activation"]) * z[:, F:]).to(dt)}
    if s["keep"]:
        out["z"] = z.to(dt)
    return out


def _plain_gated_bwd(s):
    dt, F = DTYPES[s["dtype"]], s["F"]
    g, gate, up = s["g"].float(), s["z"][:, :F].float(), s["z"][:, F:].float()
    u = torch.cat([g * up * _slope(gate, s["activation"]), g * _activation(gate, s["activation"])], 1)
    out = {"grad_x": (u @ s["w"].float()).to(dt), "grad_w": (u.t() @ s["x"].float()).to(dt)}
    if s["b"] is not None:
        out["grad_b"] = u.sum(0)
    return out


def _plain_ce(s):
    z = s["x"].float() @ s["w"].float().t()
    top = z.amax(-1)
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(-1))
    counts = s["target"] >= 0
    at = z.gather(1, s["target"].clamp(min=0)[:, None])[:, 0]
    return {"loss": torch.where(counts, lse - at, torch.zeros_like(lse)), "lse": lse}


def _plain_ce_bwd(s):
    dt = DTYPES[s["dtype"]]
    x, w = s["x"].float(), s["w"].float()
    counts = s["target"] >= 0
    g = s["g"] * counts
    d = torch.exp(x @ w.t() - s["lse"][:, None]) * (g if s["g_lse"] is None else g + s["g_lse"])[:, None]
    d[torch.arange(s["T"], device="cuda"), s["target"].clamp(min=0)] -= g
    return {"grad_x": (d @ w).to(dt), "grad_w": (d.t() @ x).to(dt)}


_PLAIN = {"gated": _plain_gated, "gated_fp8": _plain_gated, "gated_bwd": _plain_gated_bwd, "ce": _plain_ce,
          "ce_bwd": _plain_ce_bwd}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own(s):
    from invariant_mhc_aggregate_gb300 import layer
    op = s["op"]
    if op == "gated":
        if s["keep"]:
            y, z = layer.gated_linear_preact(s["x"], s["w"], bias=s["b"], activation=s["activation"])
            return {"y": y, "z": z}
        return {"y": layer.gated_linear(s["x"], s["w"], bias=s["b"], activation=s["activation"])}
    if op == "gated_fp8":
        return {"y": layer.gated_linear_fp8(s["x"], s["sx"], s["w"], s["sw"], bias=s["b"], activation=s["activation"],
                                            dtype=DTYPES[s["dtype"]])}
    if op == "gated_bwd":
        grad_x, grad_w, grad_b = layer.gated_linear_backward(s["g"], s["x"], s["w"], s["z"], activation=s["activation"],
                                                             bias=s["b"] is not None)
        out = {"grad_x": grad_x, "grad_w": grad_w}
        if grad_b is not None:
            out["grad_b"] = grad_b
        return out
    if op == "ce":
        loss, lse = layer.linear_cross_entropy(s["x"], s["w"], s["target"])
        return {"loss": loss, "lse": lse}
    grad_x, grad_w = layer.linear_cross_entropy_backward(s["g"], s["x"], s["w"], s["target"], s["lse"], grad_lse=s["g_lse"])
    return {"grad_x": grad_x, "grad_w": grad_w}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


def work(case):
    op, T, I = case["op"], case["T"], case["I"]
    if op.startswith("gated"):
        F = case["F"]
        if op == "gated_bwd":
            return {"bytes": 2 * (3 * T * F + 2 * T * I + 4 * F * I) + (8 * F if case["bias"] else 0), "flops": 8 * T * I * F}
        size = 1 if op == "gated_fp8" else 2
        return {"bytes": size * (T * I + 2 * F * I) + 2 * T * F * (3 if case["keep"] else 1) + (8 * F if case["bias"] else 0)
                + (4 * (T + 2 * F) if op == "gated_fp8" else 0), "flops": 4 * T * I * F}
    V = case["V"]
    if op == "ce":
        return {"bytes": 2 * (T * I + V * I) + 16 * T, "flops": 2 * T * I * V}
    # the logits again, then both gradients
    return {"bytes": 4 * (T * I + V * I) + (20 if case["spread"] else 16) * T, "flops": 6 * T * I * V}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _gate64(z, kind):
    """The activation and its derivative, each by its own formula."""
    if kind == "relu":
        return z.clamp(min=0), torch.where(z > 0, 1.0, 0.0).double()
    if kind == "silu":
        p = torch.special.expit(z)
        return z * p, p + z * p * (1 - p)
    if kind == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    wide = {k: v.double() if isinstance(v, torch.Tensor) and k != "target" else v for k, v in s.items()}
    x, w = wide["x"], wide["w"]
    if op.startswith("gated"):
        F = case["F"]
        if op == "gated_bwd":
            gate, up = wide["z"].split(F, dim=1)
            value, slope = _gate64(gate, case["activation"])
            parts = (wide["g"] * up * slope, wide["g"] * value)
            out = {"grad_x": torch.einsum("tf,fi->ti", parts[0], w[:F]) + torch.einsum("tf,fi->ti", parts[1], w[F:]),
                   "grad_w": torch.cat([torch.einsum("tf,ti->fi", u, x) for u in parts])}
            if wide["b"] is not None:
                out["grad_b"] = torch.cat([torch.einsum("tf->f", u) for u in parts])
            return out
        if op == "gated_fp8":
            x, w = x * wide["sx"][:, None], w * wide["sw"][:, None]
        gate, up = torch.einsum("ti,fi->tf", x, w[:F]), torch.einsum("ti,fi->tf", x, w[F:])
        if wide["b"] is not None:
            gate, up = gate + wide["b"][:F], up + wide["b"][F:]
        out = {"y": _gate64(gate, case["activation"])[0] * up}
        if case["keep"]:
            out["z"] = torch.cat([gate, up], 1)
        return out
    target = s["target"]
    rows = torch.nonzero(target >= 0)[:, 0]
    z = torch.einsum("ti,vi->tv", x, w)
    if op == "ce":
        lse = torch.logsumexp(z, -1)
        loss = torch.zeros_like(lse)
        loss[rows] = lse[rows] - (x[rows] * w[target[rows]]).sum(-1)
        return {"loss": loss, "lse": lse}
    z.sub_(wide["lse"][:, None]).exp_()
    g = torch.zeros_like(wide["g"])
    g[rows] = wide["g"][rows]
    z.mul_((g if wide["g_lse"] is None else g + wide["g_lse"])[:, None])
    z[rows, target[rows]] -= g[rows]
    return {"grad_x": torch.einsum("tv,vi->ti", z, w), "grad_w": torch.einsum("tv,ti->vi", z, x)}
