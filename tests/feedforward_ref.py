"""Plain 64-bit forms of the feed-forward operators, and the error bounds that
the kernels are held to.

Bounds.  U is the unit roundoff of the 16-bit type (2^-8 bf16, 2^-11 fp16: half a
step, counted relative to the power of two below the value; subnormal fp16 adds
2^-25 absolutely), E = 2^-23 a float32 step.

A product of k terms: the tensor cores add 16 products to the accumulator at a
time, each time off by at most two steps of the largest sum there was, and parts
of a cut tile (152 at most) and what rounds between them add as many again:
    |dz| <= acc(k) * sum |x||w|,   acc(k) = (k / 8 + 320) E
Activations are Lipschitz with constant 1.13 (1.2 here), their slopes with 1.0
(1.2 here); the kernels evaluate both to 2^-18 of the value's size (exp and a
quotient, or erfc, with a few float32 roundings; 1 + |z| bounds a slope's terms).
Rows of layer norm: sums of c values in float32, in threads and trees, are off by
at most (c / 32 + 20) E of the sum of their sizes.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25, torch.float32: 1e-38}
E = 2.0 ** -23
EVAL = 2.0 ** -18


def acc(k):
    return (k / 8 + 320) * E


def check(got, want, bound, what=""):
    got = got.double()
    assert got.shape == want.shape, f"{what}: {tuple(got.shape)}, not {tuple(want.shape)}"
    if got.numel() == 0:
        return
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    over = (got - want).abs() - bound
    at = over.argmax()
    assert float(over.max()) <= 0, (f"{what}: value {float(got.flatten()[at]):.6e}, not {float(want.flatten()[at]):.6e}: off by "
                                    f"{float((got - want).abs().flatten()[at]):.3e}, bound {float(bound.flatten()[at]):.3e}")


def rounded(want, err, dtype):
    """The bound of a value known to `err` that is rounded to `dtype`."""
    return err + U[dtype] * (want.abs() + err) + TINY[dtype]


def act(z, kind):
    """(a(z), a'(z)) in 64 bits."""
    if kind is None:
        return z, torch.ones_like(z)
    if kind == "relu":
        return z.clamp_min(0), (z > 0).double()
    if kind == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    if kind == "gelu":
        phi = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    v = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    s = torch.sigmoid(v)
    dv = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    return z * s, s + z * s * torch.sigmoid(-v) * dv


def product(x, w, transpose):
    """(X W, the sum of the terms' sizes)"""
    w = w.double().t() if transpose else w.double()
    x = x.double()
    return x @ w, x.abs() @ w.abs()


def gated(x, wg, wu, kind, transpose, dtype):
    """{name: (value, bound)} of out, gate, up."""
    k = x.shape[1]
    (g, sg), (u, su) = product(x, wg, transpose), product(x, wu, transpose)
    dg, du = acc(k) * sg, acc(k) * su
    a, _ = act(g, kind)
    da = 1.2 * dg + EVAL * a.abs() + 2.0 ** -60
    out = a * u
    err = da * (u.abs() + du) + a.abs() * du + 2 * E * out.abs()
    return dict(out=(out, rounded(out, err, dtype)), gate=(g, rounded(g, dg, dtype)), up=(u, rounded(u, du, dtype)))


def gated_grad(d, x, wg, wu, g, u, kind, transpose, dtype, grad_dtype):
    """{name: (value, bound)} of d_gate, d_up, dx, dw_gate, dw_up from the saved gate and up."""
    d, x, g, u = d.double(), x.double(), g.double(), u.double()
    a, slope = act(g, kind)
    dg, du = d * u * slope, d * a
    eg = rounded(dg, EVAL * (d * u).abs() * (1 + slope.abs()), dtype)
    eu = rounded(du, EVAL * du.abs() + 2.0 ** -60 * d.abs(), dtype)
    wg, wu = (w.double().t() if transpose else w.double() for w in (wg, wu))
    out = dict(d_gate=(dg, eg), d_up=(du, eu))
    dx = dg @ wg.t() + du @ wu.t()
    err = (eg + acc(2 * wg.shape[1]) * (dg.abs() + eg)) @ wg.t().abs() + (eu + acc(2 * wg.shape[1]) * (du.abs() + eu)) @ wu.t().abs()
    out["dx"] = (dx, rounded(dx, err, dtype))
    for name, v, e in (("dw_gate", dg, eg), ("dw_up", du, eu)):
        out[name] = weight_grad(x, v, e, transpose, grad_dtype)
    return out


def weight_grad(x, v, e, transpose, grad_dtype):
    dw, err = x.t() @ v, x.abs().t() @ (e + acc(x.shape[0]) * (v.abs() + e))
    if transpose:
        dw, err = dw.t(), err.t()
    return dw, rounded(dw, err, grad_dtype)


def linear(x, w, bias, residual, kind, transpose, dtype):
    """{name: (value, bound)} of out, pre."""
    z, s = product(x, w, transpose)
    dz = acc(x.shape[1]) * s
    if bias is not None:
        z = z + bias.double()
        dz = dz + E * (z.abs() + dz)
    a, _ = act(z, kind)
    err = 1.2 * dz + EVAL * a.abs() + 2.0 ** -60 if kind else dz
    out = a
    if residual is not None:
        out = a + residual.double()
        err = err + E * (out.abs() + err)
    return dict(out=(out, rounded(out, err, dtype)), pre=(z, rounded(z, dz, dtype)))


def linear_grad(d, x, w, pre, kind, transpose, dtype, grad_dtype):
    """{name: (value, bound)} of dx, dw, d_bias (and d_pre) from the saved sum."""
    d, x = d.double(), x.double()
    v, e, out = d, torch.zeros_like(d), {}
    before = e
    if kind:
        _, slope = act(pre.double(), kind)
        v = d * slope
        before = EVAL * d.abs() * (1 + slope.abs())
        e = rounded(v, before, dtype)
        out["d_pre"] = (v, e)
    w = w.double().t() if transpose else w.double()
    dx = v @ w.t()
    out["dx"] = (dx, rounded(dx, (e + acc(w.shape[1]) * (v.abs() + e)) @ w.t().abs(), dtype))
    out["dw"] = weight_grad(x, v, e, transpose, grad_dtype)
    db = v.sum(0)
    # summed before it is rounded
    out["d_bias"] = (db, rounded(db, (before + (d.shape[0] / 8 + 64) * E * (v.abs() + before)).sum(0), grad_dtype))
    return out


def norm(x, weight, bias, eps, dtype):
    """{name: (value, bound)} of out, mean, rstd."""
    x = x.double()
    c = x.shape[1]
    s = (c / 32 + 20) * E
    mean = x.mean(1, keepdim=True)
    e_mean = s * x.abs().mean(1, keepdim=True)
    centred = x - mean
    var = centred.square().mean(1, keepdim=True)
    # the sum of squares about a mean that is off by e_mean, of differences that are rounded
    e_x = e_mean + E * (centred.abs() + e_mean)
    e_var = (2 * centred.abs() * e_x + e_x ** 2).mean(1, keepdim=True) + s * var
    rstd = 1 / torch.sqrt(var + eps)
    e_rstd = rstd * (e_var / (var + eps) + 4 * E)
    y = centred * rstd
    err = e_x * rstd + (centred.abs() + e_x) * e_rstd + 2 * E * y.abs()
    if weight is not None:
        y, err = y * weight.double(), err * weight.double().abs()
        err = err + E * y.abs()
    if bias is not None:
        y = y + bias.double()
        err = err + E * (y.abs() + err)
    return dict(out=(y, rounded(y, err, dtype)), mean=(mean[:, 0], e_mean[:, 0] + E * mean.abs()[:, 0]),
                rstd=(rstd[:, 0], (e_rstd + E * rstd)[:, 0]))


def norm_grad(d, x, mean, rstd, weight, add, dtype, grad_dtype):
    """{name: (value, bound)} of dx, d_weight, d_bias from the statistics that the kernel is given."""
    d, x, mean, rstd = d.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    rows, c = x.shape
    s = (c / 32 + 20) * E
    xhat = (x - mean) * rstd
    e_x = 2 * E * xhat.abs()
    g = d * weight.double() if weight is not None else d
    e_g = E * g.abs()
    mg, mgx = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    e_mg = s * g.abs().mean(1, keepdim=True)
    size = (g * xhat).abs()
    e_mgx = (s + 4 * E) * size.mean(1, keepdim=True)
    inner = g - mg - xhat * mgx
    err = e_g + e_mg + xhat.abs() * e_mgx + e_x * mgx.abs() + 4 * E * (g.abs() + mg.abs() + (xhat * mgx).abs())
    dx = rstd * inner
    err = err * rstd + E * dx.abs()
    if add is not None:
        dx = dx + add.double()
        err = err + E * (dx.abs() + err)
    dw, db = (d * xhat).sum(0), d.sum(0)
    t = (rows / 8 + 64) * E
    e_dw = ((t + 4 * E) * (d * xhat).abs()).sum(0)
    return dict(dx=(dx, rounded(dx, err, dtype)), d_weight=(dw, rounded(dw, e_dw, grad_dtype)),
                d_bias=(db, rounded(db, (t * d.abs()).sum(0), grad_dtype)))
