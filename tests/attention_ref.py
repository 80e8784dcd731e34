"""Plain 64-bit forms of the attention operators, and the error bounds that
the kernels are held to.

Bounds.  u is the unit roundoff of the 16-bit type (2^-8 bf16, 2^-11 fp16).
A rotated head is computed in float32 and rounded once: |err| <= u |y| plus a
few float32 roundings of the pair's size.  An attention output is
sum(p v) / sum(p): each weight p is rounded to 16 bits before it multiplies v
(relative error u), a score of at most 128 products is off by at most
128 * 2^-24 * scale * sum |q k| (1e-4 for heads of unit mean square; a weight is off
by as much, relatively, above and below the line), and the output is rounded
once more:
    |err| <= u |o| + (u + 5e-4) * sum(p |v|) / sum(p)
fp16 weights below 2^-14 are also off by 2^-25 absolutely, the largest being at
least 1: + n * 2^-25 * max |v| for n keys.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def rope_ref(qkv, q_weight, k_weight, positions, inv_freq, axis_of_pair, rotary_dim, adjacent, eps, q_heads, kv_heads):
    """(q, k, v, bound of q, bound of k) from [tokens, heads, d] rows on any device."""
    x = qkv.double()
    t, _, d = x.shape

    def heads(y, w):
        if w is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
        half = rotary_dim // 2
        out, size = y.clone(), y.abs()
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
            ang = positions[axis_of_pair[i]].double() * inv_freq[i]
            c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
            out[..., a] = y[..., a] * c - y[..., b] * s
            out[..., b] = y[..., b] * c + y[..., a] * s
            big = y[..., a].abs() + y[..., b].abs()
            size[..., a], size[..., b] = big, big
        # norm: about d/16 + 10 float32 roundings, rotation: a few more, sincos within 2^-22
        return out, U[qkv.dtype] * out.abs() + 40 * 2.0 ** -24 * size + 2.0 ** -25

    q, bq = heads(x[:, :q_heads], q_weight)
    k, bk = heads(x[:, q_heads:q_heads + kv_heads], k_weight)
    return q, k, x[:, q_heads + kv_heads:], bq, bk


def attend(q, k, v, seen, scale, dtype):
    """One head: q [n, d], k, v [m, d], seen [n, m]; (o, bound).  Keys and values that no row sees are not looked at."""
    n, m = seen.shape
    if m == 0:
        return torch.zeros_like(q, dtype=torch.float64), torch.zeros_like(q, dtype=torch.float64)
    s = (q.double() @ k.double().T * scale).masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top)), torch.zeros_like(s))
    total = p.sum(-1, keepdim=True)
    total = torch.where(total > 0, total, torch.ones_like(total))
    o, size = p @ v.double() / total, p @ v.double().abs() / total
    u = U[dtype]
    bound = u * o.abs() + (u + 5e-4) * size + 1e-30
    if dtype == torch.float16:
        bound = bound + (m + 1) * 2.0 ** -25 * v.double().abs().max()
    return o, bound


def check(got, want, bound, what=""):
    got = got.double()
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    over = (got - want).abs() - bound
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, f"{what}: an error is {worst:.3e} over its bound {float(bound.flatten()[over.argmax()]):.3e}"


def unit(x, std=1.0):
    f = x.float()
    return (f * (std * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-9))).to(x.dtype)
