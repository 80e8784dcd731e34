"""The feed-forward half of a transformer block, forward, backward and for one token:

    x [tokens, HIDDEN] -> layer_norm -> gated_matmul (gate, up, silu, product)
      -> linear_matmul (down product onto the residual x)

    python examples/feed_forward_block.py

The operators record nothing for autograd: each is a torch.autograd.Function of
a few lines here, with its saved tensors and its backward call.  The block's
normed rows come as SHARDS shards, as a gathered product has them.  The example
compares the gradients with those of the same block in 64 bits, and the last
token alone with its row of the batch.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import all_gather_gemm_agmm_gb300 as agmm  # noqa: E402

HIDDEN, INNER, SHARDS, EPS = 512, 1408, 4, 1e-5
NAMES = ("norm weight", "norm bias", "gate", "up", "down")


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        out, mean, rstd = agmm.layer_norm(x, weight, bias, EPS, return_stats=True)
        ctx.save_for_backward(x, mean, rstd, weight)
        return out

    @staticmethod
    def backward(ctx, d_out):
        x, mean, rstd, weight = ctx.saved_tensors
        return agmm.layer_norm_backward(d_out, x, mean, rstd, weight)


class Gated(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up):
        out, gate, up = agmm.gated_matmul(shards(x), w_gate, w_up, rhs_transpose=True, return_saved=True)
        ctx.save_for_backward(x, w_gate, w_up, gate, up)
        return out

    @staticmethod
    def backward(ctx, d_out):
        x, w_gate, w_up, gate, up = ctx.saved_tensors
        return agmm.gated_matmul_backward(d_out, shards(x), w_gate, w_up, gate, up, rhs_transpose=True)


class Down(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, residual):
        ctx.save_for_backward(x, w)
        return agmm.linear_matmul(x, w, residual=residual, rhs_transpose=True)

    @staticmethod
    def backward(ctx, d_out):
        x, w = ctx.saved_tensors
        dx, dw, _ = agmm.linear_matmul_backward(d_out, x, w, rhs_transpose=True)
        return dx, dw, d_out


def shards(x):
    """x as SHARDS shards of a gathered matrix, where its rows divide so."""
    return list(x.chunk(SHARDS)) if x.shape[0] % SHARDS == 0 else [x]


def parameters(seed=0, device="cuda", dtype=torch.bfloat16):
    g = torch.Generator(device=device).manual_seed(seed)
    new = lambda *s, std: torch.randn(s, generator=g, device=device) * std  # noqa: E731
    p = [1 + new(HIDDEN, std=0.1), new(HIDDEN, std=0.1), new(INNER, HIDDEN, std=HIDDEN ** -0.5), new(INNER, HIDDEN, std=HIDDEN ** -0.5),
         new(HIDDEN, INNER, std=INNER ** -0.5)]
    return [x.to(dtype).requires_grad_() for x in p]


def block(x, params):
    weight, bias, gate, up, down = params
    return Down.apply(Gated.apply(LayerNorm.apply(x, weight, bias), gate, up), down, x)


def block64(x, params):
    """The same in 64 bits."""
    weight, bias, gate, up, down = params
    h = torch.nn.functional.layer_norm(x, (HIDDEN,), weight, bias, EPS)
    return x + (torch.nn.functional.silu(h @ gate.t()) * (h @ up.t())) @ down.t()


def gradients(tokens, seed=1, device="cuda"):
    """{name: (the operators' gradient, the same in 64 bits)}, the output's pair first."""
    g = torch.Generator(device=device).manual_seed(seed)
    x = torch.randn((tokens, HIDDEN), generator=g, device=device).bfloat16().requires_grad_()
    d = torch.randn((tokens, HIDDEN), generator=g, device=device).bfloat16()
    params = parameters()
    y = block(x, params)
    y.backward(d)
    x64, params64 = x.detach().double().requires_grad_(), [p.detach().double().requires_grad_() for p in params]
    y64 = block64(x64, params64)
    y64.backward(d.double())
    out = {"output": (y.detach(), y64.detach()), "x": (x.grad, x64.grad)}
    out.update({n: (p.grad, q.grad) for n, p, q in zip(NAMES, params, params64)})
    return out, x.detach(), params


def main():
    pairs, x, params = gradients(256)
    for name, (a, b) in pairs.items():
        off = float((a.double() - b).norm() / b.norm())
        print(f"{name:12s} {tuple(a.shape)} off by {off:.1e} of its norm")
        assert off < 2e-2, name
    with torch.no_grad():
        alone = block(x[-1:], params)
    row = pairs["output"][0][-1:]
    off = float((alone.double() - row.double()).abs().max() / row.double().abs().max())
    print(f"one token alone: off by {off:.1e} of the largest value of its row in the batch")
    assert off < 2e-2


if __name__ == "__main__":
    main()
