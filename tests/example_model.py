"""Usage example of a gated feed-forward and a model's loss: two mHC blocks' training step (aggregate, norm, gated
product, down projection, post), then the streams' collapse, its norm and the cross entropy over a vocabulary; and a
scoring step of a few tokens with 8-bit projections.  Run by test_example_model_gpu.py on a GPU."""

import torch

from invariant_mhc_aggregate_gb300 import layer
from invariant_mhc_aggregate_gb300.autograd import (gated_linear, h_aggregate, linear, linear_cross_entropy, mhc_post,
                                                    rms_norm)

T, n, H, F, V, blocks = 320, 4, 1024, 2816, 20011, 2


def parameters(gen):
    def weight(rows, length):
        return (torch.randn(rows, length, generator=gen, device="cuda") * length ** -0.5).to(torch.bfloat16).requires_grad_()

    def ones():
        return torch.ones(H, device="cuda", requires_grad=True)

    return {"blocks": [{"norm": ones(), "gate_up": weight(2 * F, H), "down": weight(H, F)} for _ in range(blocks)],
            "norm": ones(), "vocabulary": weight(V, H)}


def coefficients(gen):
    """The mixing coefficients of every block, and those of the last collapse."""
    return [(torch.rand(T, n, generator=gen, device="cuda"), 2 * torch.rand(T, n, generator=gen, device="cuda"),
             torch.softmax(torch.randn(T, n, n, generator=gen, device="cuda"), -1)) for _ in range(blocks)], \
        torch.rand(T, n, generator=gen, device="cuda")


def train_step(p, streams, mixing, collapse, target):
    """The mean loss over the tokens that count, with a term that keeps the logits' normaliser small."""
    for block, (pre, post, res) in zip(p["blocks"], mixing):
        x = h_aggregate(streams, pre)                                    # [T,H]: n streams -> one row
        y, _ = rms_norm(x, block["norm"])
        h = gated_linear(y, block["gate_up"])                            # silu(y w_gate^T) * (y w_up^T), [T,F]
        streams = mhc_post(streams, linear(h, block["down"], residual=x), post, res)
    y, _ = rms_norm(h_aggregate(streams, collapse), p["norm"])
    loss, lse = linear_cross_entropy(y, p["vocabulary"], target)         # the [T,V] logits are never stored
    count = (target >= 0).sum()
    return (loss.sum() + 1e-4 * (lse * (target >= 0)).square().sum()) / count


def score_step(p, rows, target, w8):
    """The loss of a few tokens, with 8-bit projections."""
    block = p["blocks"][0]
    y8, scale, total, _ = layer.rms_norm_fp8(rows, block["norm"].detach())
    h = layer.gated_linear_fp8(y8, scale, *w8)
    z = layer.linear(h, block["down"].detach(), residual=total)
    y, _, _ = layer.rms_norm(z, p["norm"].detach())
    return layer.linear_cross_entropy(y, p["vocabulary"].detach(), target)[0]


def eight_bits(w):
    """E4M3 values and one scale per row of a weight."""
    scale = w.detach().float().abs().amax(-1) / 448
    return (w.detach().float() / scale[:, None]).to(torch.float8_e4m3fn), scale


def main():
    gen = torch.Generator(device="cuda").manual_seed(0)
    p = parameters(gen)
    mixing, collapse = coefficients(gen)
    streams = torch.randn(T, n, H, generator=gen, device="cuda").to(torch.bfloat16).requires_grad_()
    target = torch.randint(0, V, (T,), generator=gen, device="cuda")
    target[::5] = -100                                                   # a prompt's tokens
    loss = train_step(p, streams, mixing, collapse, target)
    loss.backward()
    rows = torch.randn(7, H, generator=gen, device="cuda").to(torch.bfloat16)
    scores = score_step(p, rows, target[1:8].clamp(min=0), eight_bits(p["blocks"][0]["gate_up"]))
    return p, mixing, collapse, streams, target, loss, rows, scores


if __name__ == "__main__":
    main()
