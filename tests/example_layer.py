"""Usage example of the layer operators: an mHC block's training step (aggregate, norm, products, rotary,
post) and a decode step with 8-bit products; run by test_example_layer_gpu.py on a GPU."""

import torch

from invariant_mhc_aggregate_gb300 import layer
from invariant_mhc_aggregate_gb300.autograd import h_aggregate, linear, mhc_post, rms_norm, rotary

T, n, H, heads, D, F = 512, 4, 2048, 16, 128, 8192


def parameters(gen):
    def weight(*shape):
        return (torch.randn(*shape, generator=gen, device="cuda") * shape[-1] ** -0.5).to(torch.bfloat16).requires_grad_()

    return {"norm": torch.ones(H, device="cuda", requires_grad=True),
            "qkv": weight(3 * heads * D, H), "qkv_bias": torch.zeros(3 * heads * D, device="cuda", requires_grad=True),
            "up": weight(F, H), "up_bias": torch.zeros(F, device="cuda", requires_grad=True), "down": weight(H, F)}


def train_step(p, streams, pre, post, res, positions, frequencies):
    """One sublayer between aggregate and post; returns the new streams and the rotated queries and keys."""
    x = h_aggregate(streams, pre)                                        # [T,H]: n streams -> one row
    y, _ = rms_norm(x, p["norm"])
    qkv = linear(y, p["qkv"], bias=p["qkv_bias"])                        # [T, 3 * heads * D]
    qk = rotary(qkv[:, :2 * heads * D].unflatten(1, (2 * heads, D)), positions, frequencies)
    z = linear(linear(y, p["up"], bias=p["up_bias"], activation="gelu"), p["down"], residual=x)
    return mhc_post(streams, z, post, res), qk                           # back onto the streams


def decode_step(p, row, carried, positions, frequencies, w8):
    """A few tokens with 8-bit operands: the sum, its norm in E4M3 with a scale per row, the products."""
    y8, scale, total, _ = layer.rms_norm_fp8(row, p["norm"].detach(), residual=carried)
    qkv = layer.linear_fp8(y8, scale, *w8["qkv"], bias=p["qkv_bias"].detach())
    qk = qkv[:, :2 * heads * D].unflatten(1, (2 * heads, D))
    layer.rotary(qk, positions, frequencies, out=qk)                     # in place, inside the product's rows
    up = layer.linear_fp8(y8, scale, *w8["up"], bias=p["up_bias"].detach(), activation="gelu")
    return layer.linear(up, p["down"].detach(), residual=total), qkv


def eight_bits(w):
    """E4M3 values and one scale per row of a weight."""
    scale = w.detach().float().abs().amax(-1) / 448
    return (w.detach().float() / scale[:, None]).to(torch.float8_e4m3fn), scale


def main():
    gen = torch.Generator(device="cuda").manual_seed(0)
    p = parameters(gen)
    streams = torch.randn(T, n, H, generator=gen, device="cuda").to(torch.bfloat16).requires_grad_()
    pre = torch.rand(T, n, generator=gen, device="cuda").requires_grad_()
    post = (2 * torch.rand(T, n, generator=gen, device="cuda")).requires_grad_()
    res = torch.softmax(torch.randn(T, n, n, generator=gen, device="cuda"), -1).requires_grad_()
    frequencies = layer.rotary_frequencies(D, scaling="yarn", factor=4.0)
    out, qk = train_step(p, streams, pre, post, res, torch.arange(T, device="cuda"), frequencies)
    (out.float().square().mean() + qk.float().square().mean()).backward()

    w8 = {k: eight_bits(p[k]) for k in ("qkv", "up")}
    row, carried = (torch.randn(3, H, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    z, qkv = decode_step(p, row, carried, torch.tensor([5, 70, 100000], device="cuda"), frequencies, w8)
    return p, streams, pre, out, qk, z, qkv, row, carried


if __name__ == "__main__":
    main()
