"""One attention layer of a serving step, from gathered rows to attention:

    shards of hidden rows --all_gather_matmul--> Q, K, V
      --NormRopePlan--> normed, rotated queries and keys; keys and values in a paged cache
      --PromptPlan--> attention of the packed prompts
    then drafted tokens of every sequence: the same product and rotation, and
      --TreePlan--> attention of the drafts over the cache

    python examples/prompt_and_drafts.py

Drafts that form a chain are the next tokens of their sequence, so their
attention must agree with that of a prompt which has them at its end: the
example checks that, and then runs a tree.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import all_gather_gemm_agmm_gb300 as agmm  # noqa: E402

Q_HEADS, KV_HEADS, DIM, HIDDEN, PAGE = 16, 4, 64, 512, 16
SHARDS = 4


def layer(seed=0, device="cuda"):
    """Weights of the layer: the QKV product's, [n, k], and the head norms'."""
    g = torch.Generator(device=device).manual_seed(seed)
    n = (Q_HEADS + 2 * KV_HEADS) * DIM
    w = (torch.randn((n, HIDDEN), generator=g, device=device) * HIDDEN ** -0.5).bfloat16()
    norm = [(1 + 0.1 * torch.randn(DIM, generator=g, device=device)).bfloat16() for _ in range(2)]
    return w, norm[0], norm[1]


class Cache:
    """Pages of keys and values, and which of them each sequence has."""

    def __init__(self, pages, sequences, pages_each, device="cuda"):
        self.k, self.v = (torch.zeros((pages, PAGE, KV_HEADS, DIM), dtype=torch.bfloat16, device=device) for _ in range(2))
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(7))[:sequences * pages_each]
        self.table = order.view(sequences, pages_each).int().to(device)

    def slots(self, sequence, places):
        """The cache slots of places of sequences (two index tensors)."""
        return self.table[sequence, places // PAGE].long() * PAGE + places % PAGE


def qkv(weights, hidden):
    """The rows' QKV product, as a rank of SHARDS sees it: gathered while multiplied."""
    pad = -hidden.shape[0] % SHARDS
    rows = torch.nn.functional.pad(hidden, (0, 0, 0, pad)).view(SHARDS, -1, HIDDEN)
    out = agmm.all_gather_matmul([r.contiguous() for r in rows], weights, my_id=0, rhs_transpose=True)
    return out[:hidden.shape[0]]


def prompts(params, hidden, lens, cache=None):
    """Attention of packed prompts; their keys and values go to the cache, when there is one."""
    w, q_norm, k_norm = params
    dev = hidden.device
    sequence = torch.repeat_interleave(torch.arange(len(lens), device=dev), torch.tensor(lens, device=dev))
    starts = torch.tensor([0] + lens, device=dev).cumsum(0).int()
    place = torch.arange(hidden.shape[0], device=dev) - starts[:-1].long()[sequence]
    rows = qkv(w, hidden)
    where = {} if cache is None else dict(k_cache=cache.k, v_cache=cache.v, slots=cache.slots(sequence, place))
    q, k = agmm.qkv_norm_rope(rows, q_norm, k_norm, place[None], Q_HEADS, KV_HEADS, **where)
    v = rows.view(-1, Q_HEADS + 2 * KV_HEADS, DIM)[:, Q_HEADS + KV_HEADS:]  # as the product left them
    return agmm.prompt_attention(q, k, v, starts)


def drafts(params, hidden, context, parents, cache, chain=False):
    """Attention of drafted tokens: parents[s][i] is the parent of draft i of sequence s (-1: the context's last token)."""
    w, q_norm, k_norm = params
    dev = hidden.device
    counts = [len(p) for p in parents]
    sequence = torch.repeat_interleave(torch.arange(len(counts), device=dev), torch.tensor(counts, device=dev))
    starts = torch.tensor([0] + counts, device=dev).cumsum(0).int()
    node = torch.arange(hidden.shape[0], device=dev) - starts[:-1].long()[sequence]
    depth = []  # a draft's position is its depth in the tree; its place in the cache, its number
    for tree in parents:
        d = []
        for p in tree:
            d.append(0 if p < 0 else d[p] + 1)
        depth += d
    context = torch.tensor(context, device=dev)
    rows = qkv(w, hidden)
    q, _ = agmm.qkv_norm_rope(rows, q_norm, k_norm, (context[sequence] + torch.tensor(depth, device=dev))[None], Q_HEADS, KV_HEADS,
                              k_cache=cache.k, v_cache=cache.v, slots=cache.slots(sequence, context[sequence] + node))
    return agmm.tree_attention(q, cache.k, cache.v, cache.table, context.int(), starts, mask=None if chain else agmm.tree_mask(parents),
                               max_nodes=max(counts))


def main():
    params = layer()
    g = torch.Generator(device="cuda").manual_seed(1)
    lens, extra = [37, 300, 5, 129], [4, 4, 4, 4]
    total = [n + e for n, e in zip(lens, extra)]
    hidden = torch.randn((sum(total), HIDDEN), generator=g, device="cuda").bfloat16()
    parts = [x.split([n, e]) for x, n, e in zip(hidden.split(total), lens, extra)]
    prompt_rows, next_rows = (torch.cat([p[i] for p in parts]) for i in (0, 1))

    cache = Cache(pages=80, sequences=len(lens), pages_each=20)
    out = prompts(params, prompt_rows, lens, cache)
    whole = prompts(params, hidden, total)
    begins = torch.cat([w[:n] for w, n in zip(whole.split(total), lens)])
    chain = drafts(params, next_rows, lens, [list(range(-1, e - 1)) for e in extra], cache, chain=True)
    ends = torch.cat([w[n:] for w, n in zip(whole.split(total), lens)])
    off = [float((a.float() - b.float()).norm() / b.float().norm()) for a, b in ((out, begins), (chain, ends))]
    print(f"prompts of {lens}: relative difference {off[0]:.1e}; {extra} drafts as a chain: {off[1]:.1e}")
    assert max(off) < 1e-2, off

    tree = drafts(params, next_rows, lens, [[-1, 0, 0, 1]] * 4, cache)
    # the first draft of each tree sees what it saw in the chain
    same = float((tree[::4].float() - chain[::4].float()).abs().max())
    print(f"trees: {tuple(tree.shape)}, roots differ from the chain's by {same:.1e}")
    assert same < 1e-2 and bool(torch.isfinite(tree).all())


if __name__ == "__main__":
    main()
