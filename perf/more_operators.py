"""The cases that time the feed-forward operators and hold them to a definition.

Three operators make the feed-forward half of a transformer block around the
gathered product of this package:

  norm    LayerNormPlan: layer norm of packed rows; its backward pass with the
          gradients of weight and bias, reduced over the tokens;
  gated   GatedPlan: act(X Wg) * (X Wu) of the gathered rows, both projections,
          the activation and the product in one kernel; its backward pass;
  linear  LinearPlan: act(X W + bias) + residual of the gathered rows in one
          kernel; its backward pass.

`run` computes them in elementary torch operations where `own` is false, and
by the package's calls where it is true.  A training case is one forward and
one backward pass.  `exact` gives the same outputs from the definitions in 64
bits.
"""
import math
import random

import torch

own = False
EPS = 1e-5


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one decoded token of one user: nothing but latency
        dict(name="norm_one_token", op="norm", tokens=1, k=4096, f16=False, train=False, bias=True, add=False),
        # a training step of a small fp16 model over a ragged batch
        dict(name="norm_ragged", op="norm", tokens=509, k=1000, f16=True, train=True, bias=True, add=False),
        # a training step over the gathered rows of 8 shards of 2048, with the residual path's gradient
        dict(name="norm_step", op="norm", tokens=16384, k=8192, f16=False, train=True, bias=True, add=True),
        # one decoded token of one user: the bandwidth of the weights
        dict(name="gated_one_token", op="gated", shards=1, rows=1, k=4096, n=7168, transpose=True, f16=False, act="silu", train=False),
        # a decode step of a batch on 4 shards
        dict(name="gated_batch", op="gated", shards=4, rows=16, k=4096, n=7168, transpose=True, f16=False, act="silu", train=False),
        # prompts on 8 shards, weights stored the other way
        dict(name="gated_prompt", op="gated", shards=8, rows=256, k=8192, n=3584, transpose=False, f16=False, act="silu", train=False),
        # a training step of a small fp16 model, ragged in every direction
        dict(name="gated_train_ragged", op="gated", shards=1, rows=1003, k=1288, n=2056, transpose=False, f16=True, act="gelu_tanh", train=True),
        # a training step over 8192 tokens: the rate of the tensor cores
        dict(name="gated_train", op="gated", shards=1, rows=8192, k=4096, n=7168, transpose=True, f16=False, act="silu", train=True),
        # one decoded token through the projection back, onto the residual
        dict(name="linear_one_token", op="linear", shards=1, rows=1, k=7168, n=4096, transpose=True, f16=False, act=None, bias=False,
             residual=True, train=False),
        # a training step of a few tokens through a small layer
        dict(name="linear_train_small", op="linear", shards=1, rows=37, k=520, n=1000, transpose=True, f16=False, act="relu", bias=True,
             residual=False, train=True),
        # long prompts through the projection back, 8 shards of 2048 rows
        dict(name="linear_prompt", op="linear", shards=8, rows=2048, k=7168, n=8192, transpose=True, f16=False, act=None, bias=True,
             residual=True, train=False),
        # a training step of a plain feed-forward layer in fp16
        dict(name="linear_train", op="linear", shards=1, rows=4096, k=2560, n=5120, transpose=False, f16=True, act="gelu", bias=True,
             residual=True, train=True),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "gated", "gated", "linear", "linear"])
    c = dict(op=op, f16=rng.random() < 0.4, train=rng.random() < 0.5)
    k = 8 * _log(rng, 8, 1024)
    if op == "norm":
        c.update(tokens=_log(rng, 1, 16384), k=k, bias=rng.random() < 0.7, add=c["train"] and rng.random() < 0.5)
        return c
    n = 8 * _log(rng, 8, 1024)
    shards = rng.choice([1, 1, 2, 3, 8])
    most = int(3.8e12 / (k * n * (4 if op == "gated" else 2) * (3 if c["train"] else 1)))
    c.update(shards=shards, rows=_log(rng, 1, max(1, min(16384, most) // shards)), k=k, n=n, transpose=rng.random() < 0.5,
             act=rng.choice(["silu", "gelu", "gelu_tanh", "relu"]))
    if op == "linear":
        c.update(bias=rng.random() < 0.6, residual=rng.random() < 0.6)
        if rng.random() < 0.5:
            c["act"] = None
    return c


def work(case):
    k, t = case["k"], case["train"]
    if case["op"] == "norm":
        m = case["tokens"]
        rows = 2 + (2 if t else 0) + (1 if case["add"] else 0)  # x, y; d_out, dx; the gradient that is added
        return dict(bytes=2 * m * k * rows + 2 * k * (1 + case["bias"]) * (2 if t else 1), flops=m * k * (20 if t else 8))
    m, n = case["shards"] * case["rows"], case["n"]
    if case["op"] == "gated":
        elements = m * k + 2 * k * n + m * n
        return dict(bytes=2 * elements * (2 if t else 1), flops=4 * m * k * n * (3 if t else 1))
    elements = m * k + k * n + m * n + case["bias"] * n
    return dict(bytes=2 * (elements * (2 if t else 1) + case["residual"] * m * n), flops=2 * m * k * n * (3 if t else 1))


# -------------------------------------------------------------------- the inputs
class State:
    pass


def prepare(case, seed):
    s = State()
    s.case = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = torch.float16 if case["f16"] else torch.bfloat16
    k, train = case["k"], case["train"]

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std + mean).to(dt)

    def empty(*shape, dtype=dt):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if own:
        import all_gather_gemm_agmm_gb300 as agmm
    if case["op"] == "norm":
        m = case["tokens"]
        s.x = normal(m, k, std=1.5, mean=0.3)
        s.weight = normal(k, std=0.2, mean=1.0)
        s.bias = normal(k, std=0.2) if case["bias"] else None
        s.d_out = normal(m, k) if train else None
        s.add = normal(m, k) if case["add"] else None
        if own:
            s.plan = agmm.LayerNormPlan(k, eps=EPS, f16=case["f16"])
            s.out = empty(m, k)
            if train:
                s.workspace = s.plan.new_workspace()
                s.mean, s.rstd = (empty(m, dtype=torch.float32) for _ in range(2))
                s.dx, s.d_weight = empty(m, k), empty(k)
                s.d_bias = empty(k) if case["bias"] else None
        return s
    p, rows, n = case["shards"], case["rows"], case["n"]
    m = p * rows
    shape = (n, k) if case["transpose"] else (k, n)
    s.xs = [normal(rows, k) for _ in range(p)]
    s.d_out = normal(m, n) if train else None
    if case["op"] == "gated":
        s.w_gate, s.w_up = (normal(*shape, std=0.02) for _ in range(2))
        if own:
            s.plan = agmm.GatedPlan(k, n, activation=case["act"], rhs_transpose=case["transpose"], f16=case["f16"])
            s.workspace = s.plan.new_workspace()
            s.out = empty(m, n)
            s.gate = s.up = None
            if train:
                s.gate, s.up, s.d_gate, s.d_up = (empty(m, n) for _ in range(4))
                s.dx, s.dw_gate, s.dw_up = empty(m, k), empty(*shape), empty(*shape)
        return s
    s.w = normal(*shape, std=0.02)
    s.bias = normal(n, std=0.5) if case["bias"] else None
    s.residual = normal(m, n) if case["residual"] else None
    if own:
        s.plan = agmm.LinearPlan(k, n, activation=case["act"], rhs_transpose=case["transpose"], f16=case["f16"])
        s.workspace = s.plan.new_workspace()
        s.out = empty(m, n)
        s.pre = s.d_pre = s.d_bias = None
        if train:
            s.dx, s.dw = empty(m, k), empty(*shape)
            if case["act"]:
                s.pre, s.d_pre = empty(m, n), empty(m, n)
            if case["bias"]:
                s.d_bias = empty(n)
    return s


# --------------------------------------------------------------- the plain forms
def _act(z, kind):
    """The activation and its derivative."""
    if kind is None:
        return z, torch.ones_like(z)
    if kind == "relu":
        on = (z > 0).to(z.dtype)
        return z * on, on
    if kind == "silu":
        p = 1 / (1 + torch.exp(-z))
        return z * p, p * (1 + z * (1 - p))
    if kind == "gelu":
        p = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * p, p + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    inner = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * inner


def _plain_norm(s):
    c, dt = s.case, s.x.dtype
    x, w = s.x.float(), s.weight.float()
    x = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    x = x * rstd
    y = x * w
    if c["bias"]:
        y = y + s.bias.float()
    out = dict(out=y.to(dt))
    if c["train"]:
        d = s.d_out.float()
        out["d_weight"] = (d * x).sum(0).to(dt)
        if c["bias"]:
            out["d_bias"] = d.sum(0).to(dt)
        d = d * w
        dx = (d - d.mean(-1, keepdim=True) - x * (d * x).mean(-1, keepdim=True)) * rstd
        if c["add"]:
            dx = dx + s.add.float()
        out["dx"] = dx.to(dt)
    return out


def _plain_product(s):
    c = s.case
    x = torch.cat(s.xs).float()
    dt = s.xs[0].dtype
    canon = lambda w: w.float().t() if c["transpose"] else w.float()  # noqa: E731
    stored = lambda w: (w.t() if c["transpose"] else w).to(dt).contiguous()  # noqa: E731
    if c["op"] == "gated":
        wg, wu = canon(s.w_gate), canon(s.w_up)
        gate, up = x @ wg, x @ wu
        a, slope = _act(gate, c["act"])
        out = dict(out=(a * up).to(dt))
        if c["train"]:
            d = s.d_out.float()
            d_gate, d_up = d * up * slope, d * a
            out["dx"] = (d_gate @ wg.t() + d_up @ wu.t()).to(dt)
            out["dw_gate"], out["dw_up"] = stored(x.t() @ d_gate), stored(x.t() @ d_up)
        return out
    w = canon(s.w)
    z = x @ w
    if c["bias"]:
        z = z + s.bias.float()
    a, slope = _act(z, c["act"])
    if c["residual"]:
        a = a + s.residual.float()
    out = dict(out=a.to(dt))
    if c["train"]:
        d = s.d_out.float() * slope
        out["dx"], out["dw"] = (d @ w.t()).to(dt), stored(x.t() @ d)
        if c["bias"]:
            out["d_bias"] = d.sum(0).to(dt)
    return out


def run(s):
    c = s.case
    if not own:
        return _plain_norm(s) if c["op"] == "norm" else _plain_product(s)
    if c["op"] == "norm":
        if not c["train"]:
            s.plan.run(s.x, s.out, weight=s.weight, bias=s.bias)
            return dict(out=s.out)
        s.plan.run(s.x, s.out, weight=s.weight, bias=s.bias, mean=s.mean, rstd=s.rstd)
        s.plan.backward(s.d_out, s.x, s.mean, s.rstd, s.dx, s.workspace, weight=s.weight, add=s.add, d_weight=s.d_weight,
                        d_bias=s.d_bias)
        out = dict(out=s.out, d_weight=s.d_weight)
        if c["bias"]:
            out["d_bias"] = s.d_bias
        out["dx"] = s.dx
        return out
    if c["op"] == "gated":
        s.plan.run(s.xs, s.w_gate, s.w_up, s.out, s.workspace, gate=s.gate, up=s.up)
        if not c["train"]:
            return dict(out=s.out)
        s.plan.backward(s.d_out, s.xs, s.w_gate, s.w_up, s.gate, s.up, s.d_gate, s.d_up, s.workspace, dx=s.dx, dw_gate=s.dw_gate,
                        dw_up=s.dw_up)
        return dict(out=s.out, dx=s.dx, dw_gate=s.dw_gate, dw_up=s.dw_up)
    s.plan.run(s.xs, s.w, s.out, s.workspace, bias=s.bias, residual=s.residual, pre=s.pre)
    if not c["train"]:
        return dict(out=s.out)
    s.plan.backward(s.d_out, s.xs, s.w, s.workspace, pre=s.pre, d_pre=s.d_pre, dx=s.dx, dw=s.dw, d_bias=s.d_bias)
    out = dict(out=s.out, dx=s.dx, dw=s.dw)
    if c["bias"]:
        out["d_bias"] = s.d_bias
    return out


# -------------------------------------------------------- the definition, in 64 bits
def _activation(kind):
    f = torch.nn.functional
    return {None: lambda z: z, "relu": f.relu, "silu": f.silu, "gelu": f.gelu, "gelu_tanh": lambda z: f.gelu(z, approximate="tanh")}[kind]


def exact(case, seed):
    if work(case)["flops"] > 1.2e13:
        return None
    s = prepare(case, seed)
    train = case["train"]

    def leaf(x):
        return None if x is None else x.double().requires_grad_(train)

    if case["op"] == "norm":
        x, w, b = leaf(s.x), leaf(s.weight), leaf(s.bias)
        var, mean = torch.var_mean(x, -1, keepdim=True, correction=0)
        y = (x - mean) / torch.sqrt(var + EPS) * w + (0 if b is None else b)
        leaves = dict(d_weight=w, d_bias=b, dx=x)
    elif case["op"] == "gated":
        x, w, v = leaf(torch.cat(s.xs)), leaf(s.w_gate), leaf(s.w_up)
        product = lambda y: torch.einsum("mk,nk->mn" if case["transpose"] else "mk,kn->mn", x, y)  # noqa: E731
        y = _activation(case["act"])(product(w)) * product(v)
        leaves = dict(dx=x, dw_gate=w, dw_up=v)
    else:
        x, w, b = leaf(torch.cat(s.xs)), leaf(s.w), leaf(s.bias)
        z = torch.einsum("mk,nk->mn" if case["transpose"] else "mk,kn->mn", x, w)
        y = _activation(case["act"])(z if b is None else z + b)
        if s.residual is not None:
            y = y + s.residual.double()
        leaves = dict(dx=x, dw=w, d_bias=b)
    out = dict(out=y.detach())
    if train:
        y.backward(s.d_out.double())
        for name, x in leaves.items():
            if x is not None:
                out[name] = x.grad
        if case["op"] == "norm" and s.add is not None:
            out["dx"] = out["dx"] + s.add.double()
    return out
