"""The cases that time the attention operators and hold them to a definition.

Three operators stand behind the column-parallel QKV product of this package:

  norm_rope  NormRopePlan.run: RMS norm of every query and key head and the
             rotation by the token's position (one or several position axes),
             queries and keys in packed rows, keys and values into cache slots;
  prompt     PromptPlan.run: causal attention of packed prompts with grouped
             heads (a prompt may be the last piece of a longer context);
  tree       TreePlan.run: attention of drafted tokens (a tree, or one token)
             over a paged cache.

`run` computes them in elementary torch operations where `own` is false, and
by the package's calls where it is true.  `exact` gives the same outputs from
the definitions in 64 bits.
"""
import math
import random

import torch

own = False
EPS = 1e-6
BASE = 1e6


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one decoded token of one user: nothing but latency
        dict(name="rope_one_token", op="norm_rope", tokens=1, q_heads=32, kv_heads=8, dim=128, axes=1, f16=False,
             packed_k=False, cache=True, page=16, top=30000),
        # a step of drafted tokens of an image model with small heads; some tokens are padding and reach no slot
        dict(name="rope_drafts", op="norm_rope", tokens=509, q_heads=16, kv_heads=2, dim=64, axes=3, f16=True,
             packed_k=False, cache=True, page=32, top=8000),
        # a step of long prompts with images, 8 shards of 2048 rows each: the bandwidth of the memory
        dict(name="rope_prompts", op="norm_rope", tokens=16384, q_heads=64, kv_heads=8, dim=128, axes=3, f16=False,
             packed_k=True, cache=True, page=64, top=32000),
        # many short chat turns packed together, odd lengths, one of a single token
        dict(name="prompt_short_turns", op="prompt", batch=24, shortest=1, longest=333, prefix=0, q_heads=32, kv_heads=8,
             dim=128, f16=False, spread=3),
        # prompts of very different lengths, small fp16 heads
        dict(name="prompt_mixed", op="prompt", batch=5, shortest=17, longest=4001, prefix=0, q_heads=16, kv_heads=2,
             dim=64, f16=True, spread=5),
        # the next 1024 tokens or so of two documents whose beginnings are there already
        dict(name="prompt_piece", op="prompt", batch=2, shortest=700, longest=1024, prefix=15000, q_heads=32, kv_heads=8,
             dim=128, f16=False, spread=7),
        # one long document in one piece: the rate of the tensor cores
        dict(name="prompt_document", op="prompt", batch=1, shortest=8191, longest=8191, prefix=0, q_heads=32, kv_heads=8,
             dim=128, f16=False, spread=1),
        # one decoded token of one user over a short context, small pages
        dict(name="tree_one_token", op="tree", batch=1, nodes=1, shortest=1000, longest=1000, q_heads=32, kv_heads=8,
             dim=128, page=16, f16=False, spread=1),
        # a batch of users, one token each: the bandwidth of the memory
        dict(name="tree_batch", op="tree", batch=32, nodes=1, shortest=150, longest=8100, q_heads=64, kv_heads=8,
             dim=128, page=64, f16=False, spread=2),
        # small trees of a small fp16 model
        dict(name="tree_small_heads", op="tree", batch=8, nodes=24, shortest=1, longest=4111, q_heads=16, kv_heads=2,
             dim=64, page=32, f16=True, spread=4),
        # large trees over long contexts: more rows than one tile holds
        dict(name="tree_large", op="tree", batch=4, nodes=64, shortest=20000, longest=32000, q_heads=32, kv_heads=8,
             dim=128, page=128, f16=False, spread=6),
        # a few drafted tokens over the longest context
        dict(name="tree_long_context", op="tree", batch=2, nodes=5, shortest=100000, longest=131000, q_heads=32, kv_heads=8,
             dim=128, page=64, f16=False, spread=8),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))
    v = max(lo, min(hi, v))
    return v + 1 if v == 3072 else v


def _heads(rng):
    return rng.choice([(32, 8, 128), (64, 8, 128), (16, 2, 64), (40, 8, 128), (28, 4, 128), (8, 8, 64), (16, 1, 128)])


def draw(rng):
    op = rng.choice(["norm_rope", "prompt", "tree"])
    hq, hk, d = _heads(rng)
    c = dict(op=op, q_heads=hq, kv_heads=hk, dim=d, f16=rng.random() < 0.4)
    if op == "norm_rope":
        packed = rng.random() < 0.5
        c.update(tokens=_log(rng, 1, 16384), axes=rng.choice([1, 3]), packed_k=packed,
                 cache=not packed or rng.random() < 0.5, page=rng.choice([16, 32, 64, 128]), top=_log(rng, 200, 32000))
    elif op == "prompt":
        batch = _log(rng, 1, 24)
        longest = _log(rng, 8, int(8191 / math.sqrt(batch)))
        prefix = 0 if rng.random() < 0.6 else _log(rng, 1, max(1, min(15000, 8191 * 8191 // (batch * longest) - longest)))
        if batch * hq * longest * (longest + prefix) > 32 * 8191 * 8191:
            longest, prefix = max(1, longest // 2), prefix // 2
        c.update(batch=batch, shortest=_log(rng, 1, longest), longest=longest, prefix=prefix, spread=rng.randrange(1 << 20))
    else:
        batch = _log(rng, 1, 32)
        longest = _log(rng, 8, 262000 // batch)
        nodes = 1 if rng.random() < 0.4 else _log(rng, 2, 64)
        if batch * hq * nodes * longest > 4 * 32 * 64 * 32000:
            nodes = max(1, 4 * 32 * 64 * 32000 // (batch * hq * longest))
        c.update(batch=batch, nodes=nodes, shortest=_log(rng, 1, longest), longest=longest,
                 page=rng.choice([16, 32, 64, 128]), spread=rng.randrange(1 << 20))
    return c


def _lengths(case):
    """Each sequence's length (its context's, for trees): the longest is there, the others lie between the bounds."""
    r = random.Random(case["spread"])
    lens = [_log(r, case["shortest"], case["longest"]) for _ in range(case["batch"])]
    lens[0], lens[-1] = case["shortest"], case["longest"]
    r.shuffle(lens)
    return lens


def _prefixes(case):
    """How much context each prompt has before its own first token."""
    r = random.Random(case["spread"] + 1)
    return [_log(r, (case["prefix"] + 1) // 2, case["prefix"]) if case["prefix"] else 0 for _ in range(case["batch"])]


def work(case):
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "norm_rope":
        t = case["tokens"]
        rows = (hq + (hk if case["packed_k"] else 0)) + (2 * hk if case["cache"] else 0)
        read = hq + hk + (hk if case["cache"] else 0)
        return dict(bytes=2 * t * d * (read + rows) + t * (8 * case["axes"] + (8 if case["cache"] else 0)) + 4 * d,
                    flops=t * (hq + hk) * d * 8)
    if case["op"] == "prompt":
        lens, pre = _lengths(case), _prefixes(case)
        pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(lens, pre))
        return dict(bytes=2 * d * sum(2 * n * hq + 2 * (n + p) * hk for n, p in zip(lens, pre)), flops=4 * hq * d * pairs)
    ctx, n = _lengths(case), case["nodes"]
    return dict(bytes=2 * d * sum(2 * n * hq + 2 * (c + n) * hk for c in ctx), flops=4 * hq * d * sum(n * (c + 1) for c in ctx))


# -------------------------------------------------------------------- the inputs
class State:
    pass


def _randn(g, *shape, dtype, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _unit(x, std):
    """Heads as a norm leaves them: every head's mean square is std^2."""
    f = x.float()
    return (f * (std * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS))).to(x.dtype)


def _sections(case):
    half = case["dim"] // 2
    return (half,) if case["axes"] == 1 else (half - 2 * (3 * half // 8), 3 * half // 8, 3 * half // 8)


def _positions(case, rng):
    """[axes, tokens]: text moves all axes together; an image holds the first and counts rows and columns."""
    t, top = case["tokens"], case["top"]
    at = rng.randrange(top)
    if case["axes"] == 1:
        return [[(at + i) % top for i in range(t)]]
    pos = [[], [], []]
    while len(pos[0]) < t:
        if rng.random() < 0.5:
            n = rng.randrange(1, 300)
            for p in pos:
                p.extend((at + i) % top for i in range(n))
            at += n
        else:
            w, h = rng.randrange(2, 40), rng.randrange(2, 40)
            pos[0].extend([at % top] * (w * h))
            pos[1].extend((at + i) % top for i in range(h) for _ in range(w))
            pos[2].extend((at + j) % top for _ in range(h) for j in range(w))
            at += max(w, h)
    return [p[:t] for p in pos]


def _tree(n, rng):
    """The mask of a random tree of n nodes: bit j of word j / 64 of row i says that i sees j."""
    words, rows = (n + 63) // 64, []
    for i in range(n):
        parent = -1 if i == 0 else max(-1, i - 1 - min(rng.randrange(8), rng.randrange(8)))
        rows.append((rows[parent] if parent >= 0 else 0) | 1 << i)
    signed = lambda v: v - (1 << 64) if v >> 63 else v  # noqa: E731
    return [[signed(r >> 64 * w & (1 << 64) - 1) for w in range(words)] for r in rows]


def prepare(case, seed):
    s, rng = State(), random.Random(seed)
    s.case = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    dt = torch.float16 if case["f16"] else torch.bfloat16
    ints = lambda v, t=torch.int32: torch.tensor(v, dtype=t, device="cuda")  # noqa: E731
    if case["op"] == "norm_rope":
        t = case["tokens"]
        s.qkv = _randn(g, t, (hq + 2 * hk) * d, dtype=dt, std=1.7)
        s.q_weight = (1.2 + 0.3 * _randn(g, d, dtype=torch.float32)).to(dt)
        s.k_weight = (1.0 + 0.3 * _randn(g, d, dtype=torch.float32)).to(dt)
        s.positions = ints(_positions(case, rng), torch.int64)
        s.inv_freq = BASE ** (-torch.arange(d // 2, dtype=torch.float64, device="cuda") / (d // 2))
        axis = [a for a, n in enumerate(_sections(case)) for _ in range(n)]
        s.axis = ints(axis, torch.int64)
        s.q = torch.empty((t, hq, d), dtype=dt, device="cuda")
        s.k = torch.empty((t, hk, d), dtype=dt, device="cuda") if case["packed_k"] else None
        s.k_cache = s.v_cache = s.slots = None
        if case["cache"]:
            pages = -(-t // case["page"]) + 3
            s.k_cache = torch.zeros((pages, case["page"], hk, d), dtype=dt, device="cuda")
            s.v_cache = torch.zeros((pages, case["page"], hk, d), dtype=dt, device="cuda")
            order = torch.randperm(pages * case["page"], generator=g, device="cuda")[:t]
            s.slots = torch.where(torch.rand(t, generator=g, device="cuda") < 0.01, -1, order) if t > 1 else order
        if own:
            import all_gather_gemm_agmm_gb300 as agmm

            s.plan = agmm.NormRopePlan(hq, hk, d, sections=_sections(case), base=BASE, eps=EPS, f16=case["f16"])
        return s
    s.scale = d ** -0.5
    if case["op"] == "prompt":
        lens, pre = _lengths(case), _prefixes(case)
        s.starts = ints([0] + [sum(lens[: i + 1]) for i in range(len(lens))])
        kv = [n + p for n, p in zip(lens, pre)]
        s.kv_starts = ints([0] + [sum(kv[: i + 1]) for i in range(len(kv))]) if any(pre) else s.starts
        s.most, s.kv_most = max(lens), max(kv)
        if any(pre):  # the keys of the whole contexts, apart from the new tokens' queries
            s.q = _unit(_randn(g, sum(lens), hq, d, dtype=dt), 1.3)
            k, s.v = (_randn(g, sum(kv), hk, d, dtype=dt) for _ in range(2))
            s.k = _unit(k, 1.0)
        else:  # all in the rows of one product, rotated in place
            rows = _randn(g, sum(lens), hq + 2 * hk, d, dtype=dt)
            rows[:, :hq] = _unit(rows[:, :hq], 1.3)
            rows[:, hq:hq + hk] = _unit(rows[:, hq:hq + hk], 1.0)
            s.q, s.k, s.v = rows[:, :hq], rows[:, hq:hq + hk], rows[:, hq + hk:]
        s.out = torch.empty((sum(lens), hq, d), dtype=dt, device="cuda")
        if own:
            import all_gather_gemm_agmm_gb300 as agmm

            s.plan = agmm.PromptPlan(hq, hk, d, f16=case["f16"])
            s.workspace = s.plan.new_workspace()
        return s
    ctx, n, page = _lengths(case), case["nodes"], case["page"]
    need = [-(-(c + n) // page) for c in ctx]
    pages = sum(need) + 5
    order = list(range(pages))
    rng.shuffle(order)
    table, at = [], 0
    for m in need:
        table.append(order[at:at + m] + [0] * (max(need) - m))
        at += m
    s.table, s.ctx = ints(table), ints(ctx)
    s.starts = ints([n * i for i in range(len(ctx) + 1)])
    s.k_cache = _unit(_randn(g, pages, page, hk, d, dtype=dt), 1.0)
    s.v_cache = _randn(g, pages, page, hk, d, dtype=dt)
    s.q = _unit(_randn(g, n * len(ctx), hq, d, dtype=dt), 1.3)
    s.mask = ints([row for _ in ctx for row in _tree(n, rng)], torch.int64) if n > 1 else None
    s.out = torch.empty_like(s.q)
    if own:
        import all_gather_gemm_agmm_gb300 as agmm

        s.plan = agmm.TreePlan(hq, hk, d, page_size=page, max_nodes=n, f16=case["f16"])
        s.workspace = s.plan.new_workspace()
    return s


# --------------------------------------------------------------- the plain forms
def _plain_rope(s):
    c = s.case
    hq, hk, d, t = c["q_heads"], c["kv_heads"], c["dim"], c["tokens"]
    x = s.qkv.view(t, hq + 2 * hk, d).float()
    qk, v = x[:, :hq + hk], x[:, hq + hk:]
    qk = qk * torch.rsqrt(qk.square().mean(-1, keepdim=True) + EPS)
    qk = torch.cat([qk[:, :hq] * s.q_weight.float(), qk[:, hq:] * s.k_weight.float()], 1)
    angle = s.positions[s.axis].t().float() * s.inv_freq.float()
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    a, b = qk[..., :d // 2], qk[..., d // 2:]
    qk = torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(s.qkv.dtype)
    out = dict(q=qk[:, :hq].contiguous())
    if c["packed_k"]:
        out["k"] = qk[:, hq:].contiguous()
    if c["cache"]:
        kept = s.slots >= 0
        s.k_cache.view(-1, hk, d)[s.slots[kept]] = qk[:, hq:][kept]
        s.v_cache.view(-1, hk, d)[s.slots[kept]] = v[kept].to(s.qkv.dtype)
        out["k_cache"], out["v_cache"] = s.k_cache, s.v_cache
    return out


def _softmax_sum(q, k, v, seen, scale):
    """q [b, q, h * g, d], k and v [b, k, h, d], seen [b, q, k] or one that spreads to it: a row that sees nothing is 0."""
    b, n, hq, d = q.shape
    h = k.shape[2]
    q = q.float().view(b, n, h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(b, h, hq // h * n, d)
    p = torch.matmul(q, k.float().permute(0, 2, 3, 1)).view(b, h, hq // h, n, -1)
    p.mul_(scale).masked_fill_(~seen[:, None, None], -math.inf)
    p.sub_(p.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, h, hq // h * n, -1), v.float().permute(0, 2, 1, 3)).view(b, h, hq // h, n, d)
    o = o / torch.where(total > 0, total, 1)
    return o.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d)


def _plain_prompt(s):
    qn, kn = s.starts.diff()[:, None], s.kv_starts.diff()[:, None]
    i, j = torch.arange(s.most, device="cuda"), torch.arange(s.kv_most, device="cuda")
    rows, cols = s.starts[:-1, None] + i, s.kv_starts[:-1, None] + j
    real = i < qn
    seen = (j[None, None] <= (i + kn - qn)[:, :, None]) & (j < kn)[:, None]
    cols = cols.clamp_max(s.k.shape[0] - 1)
    o = _softmax_sum(s.q[rows.clamp_max(s.q.shape[0] - 1)], s.k[cols], s.v[cols], seen, s.scale)
    return o[real].to(s.q.dtype)


def _plain_tree(s):
    c = s.case
    n, b = c["nodes"], c["batch"]
    k, v = (x[s.table.long()].flatten(1, 2) for x in (s.k_cache, s.v_cache))
    j = torch.arange(k.shape[1], device="cuda")
    node = j - s.ctx[:, None]  # which drafted token a place holds
    if s.mask is None:
        seen = (node <= 0)[:, None]
    else:
        words = s.mask.view(b, n, -1)
        near = node.clamp(0, n - 1).long()
        bits = words.gather(2, (near // 64)[:, None].expand(b, n, -1)) >> (near % 64)[:, None] & 1
        seen = (node < 0)[:, None] | (bits != 0) & (node < n)[:, None] & (node >= 0)[:, None]
    o = _softmax_sum(s.q.view(b, n, *s.q.shape[1:]), k, v, seen, s.scale)
    return o.flatten(0, 1).to(s.q.dtype)


def run(s):
    c = s.case
    if not own:
        return _plain_rope(s) if c["op"] == "norm_rope" else _plain_prompt(s) if c["op"] == "prompt" else _plain_tree(s)
    if c["op"] == "norm_rope":
        s.plan.run(s.qkv, s.q_weight, s.k_weight, s.positions, s.q, k=s.k, k_cache=s.k_cache, v_cache=s.v_cache, slots=s.slots)
        out = dict(q=s.q)
        if c["packed_k"]:
            out["k"] = s.k
        if c["cache"]:
            out["k_cache"], out["v_cache"] = s.k_cache, s.v_cache
        return out
    if c["op"] == "prompt":
        s.plan.run(s.q, s.k, s.v, s.starts, s.out, s.workspace, kv_starts=s.kv_starts)
    else:
        s.plan.run(s.q, s.k_cache, s.v_cache, s.table, s.ctx, s.starts, s.out, s.workspace, mask=s.mask)
    return s.out


# -------------------------------------------------------- the definition, in 64 bits
def _attend(q, k, v, seen, scale):
    """One head: q [n, d], k and v [m, d] in 64 bits, seen [n, m]; a row that sees nothing is 0."""
    w = (q @ k.T * scale).masked_fill(~seen, -math.inf)
    return torch.nan_to_num(torch.softmax(w, -1)) @ v


def exact(case, seed):
    if work(case)["flops"] > 3e12:
        return None
    s = prepare(case, seed)
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "norm_rope":
        x = s.qkv.double().view(case["tokens"], -1, d)
        half = d // 2
        turn = torch.empty((case["tokens"], half), dtype=torch.float64, device="cuda")
        for i, a in enumerate(s.axis.tolist()):
            turn[:, i] = s.positions[a].double() * BASE ** (-i / half)

        def rotated(heads, weight):
            y = heads / (heads.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * weight.double()
            z = torch.complex(y[..., :half], y[..., half:]) * torch.polar(torch.ones_like(turn), turn)[:, None]
            return torch.cat([z.real, z.imag], -1)

        q, k, v = rotated(x[:, :hq], s.q_weight), rotated(x[:, hq:hq + hk], s.k_weight), x[:, hq + hk:]
        out = dict(q=q)
        if case["packed_k"]:
            out["k"] = k
        if case["cache"]:
            places = s.k_cache.shape[0] * case["page"]
            caches = torch.zeros((2, places + 1, hk, d), dtype=torch.float64, device="cuda")
            at = torch.where(s.slots < 0, places, s.slots)
            caches[0, at], caches[1, at] = k, v
            out["k_cache"], out["v_cache"] = (c[:places].view(-1, case["page"], hk, d) for c in caches)
        return out
    q, g = s.q.double(), hq // hk
    out = torch.zeros_like(q)
    if case["op"] == "prompt":
        at, kv_at = s.starts.tolist(), s.kv_starts.tolist()
        for b in range(case["batch"]):
            rows, cols = slice(at[b], at[b + 1]), slice(kv_at[b], kv_at[b + 1])
            n, m = at[b + 1] - at[b], kv_at[b + 1] - kv_at[b]
            seen = torch.ones((n, m), dtype=torch.bool, device="cuda").tril(m - n)
            for h in range(hq):
                out[rows, h] = _attend(q[rows, h], s.k[cols, h // g].double(), s.v[cols, h // g].double(), seen, s.scale)
        return out
    n, page = case["nodes"], case["page"]
    for b, c in enumerate(s.ctx.tolist()):
        place = torch.arange(c + n, device="cuda")
        pages, within = s.table[b].long()[place // page], place % page
        seen = torch.ones((n, c + n), dtype=torch.bool, device="cuda")
        for i in range(n):
            for j in range(n):
                seen[i, c + j] = i == j if s.mask is None else False
        if s.mask is not None:
            words = s.mask[n * b:n * b + n].tolist()
            seen[:, c:] = torch.tensor([[bool(words[i][j // 64] >> j % 64 & 1) for j in range(n)] for i in range(n)], device="cuda")
        for h in range(hk):
            k, v = (x[pages, within, h].double() for x in (s.k_cache, s.v_cache))
            rows = q[n * b:n * b + n, g * h:g * h + g]
            o = _attend(rows.reshape(n * g, d), k, v, seen.repeat_interleave(g, 0), s.scale)
            out[n * b:n * b + n, g * h:g * h + g] = o.view(n, g, d)
    return out
