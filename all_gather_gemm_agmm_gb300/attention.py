"""The operators behind a column-parallel QKV product: head norms with rotary
positions, attention of packed prompts, attention of drafted tokens over a
paged cache.

Every step of the computation runs in the CUDA kernels of ``libagmm.so``
(``include/agmm_attention.h``, which defines each operator); this module
checks arguments and marshals them.  PyTorch supplies device memory and
streams.  There is no CPU fallback.

As with :class:`Plan`, a plan is made once for a layer's shape and its ``run``
takes the caller's buffers; the functions ``qkv_norm_rope``,
``prompt_attention`` and ``tree_attention`` allocate them.  Buffers follow
PyTorch's stream rules: a tensor used on a ``stream`` other than the one it
was made on has to be ready there, and to outlive the work.  A ``stream`` is a
``torch.cuda.Stream``, an object with a ``cuda_stream`` handle, or the handle;
what the functions allocate belongs to it.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Dict, List, Optional, Sequence

from . import AGMM_BF16, AGMM_F16, _check, _On, load_library

ATTENTION_SYMBOLS = [
    "agmm_norm_rope_plan", "agmm_norm_rope_run", "agmm_norm_rope_destroy",
    "agmm_prompt_plan", "agmm_prompt_workspace_bytes", "agmm_prompt_run", "agmm_prompt_destroy",
    "agmm_tree_plan", "agmm_tree_workspace_bytes", "agmm_tree_run", "agmm_tree_destroy",
]


class _NormRopeDesc(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in ("q_heads", "kv_heads", "head_dim", "rotary_dim", "adjacent", "axes", "dtype")]
    _fields_ += [("eps", ctypes.c_float), ("inv_freq", ctypes.POINTER(ctypes.c_double)),
                 ("axis_of_pair", ctypes.POINTER(ctypes.c_int))]


class _PromptDesc(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in ("q_heads", "kv_heads", "head_dim", "causal", "dtype")]
    _fields_ += [("scale", ctypes.c_float)]


class _TreeDesc(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in ("q_heads", "kv_heads", "head_dim", "page_size", "max_nodes", "dtype")]
    _fields_ += [("scale", ctypes.c_float)]


# The *_args_t structs are 64-bit fields throughout, packed in one step.
_NORM_ROPE_ARGS = struct.Struct("=23q")
_PROMPT_ARGS = struct.Struct("=18q")
_TREE_ARGS = struct.Struct("=22q")

MAX_NODES = 1024  # what agmm_tree_plan takes

_bound = None


def _library() -> ctypes.CDLL:
    """libagmm.so with the signatures of agmm_attention.h declared."""
    global _bound
    if _bound is not None:
        return _bound
    lib = load_library()
    vp, c_int, out = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(ctypes.c_void_p)
    for name, desc in (("norm_rope", _NormRopeDesc), ("prompt", _PromptDesc), ("tree", _TreeDesc)):
        f = getattr(lib, f"agmm_{name}_plan")
        f.argtypes, f.restype = [ctypes.POINTER(desc), out], c_int
        f = getattr(lib, f"agmm_{name}_run")
        f.argtypes, f.restype = [vp, ctypes.c_char_p, vp], c_int
        f = getattr(lib, f"agmm_{name}_destroy")
        f.argtypes, f.restype = [vp], None
        if name != "norm_rope":
            f = getattr(lib, f"agmm_{name}_workspace_bytes")
            f.argtypes, f.restype = [vp], ctypes.c_size_t
    _bound = lib
    return lib


class _AttentionPlan:
    """What the three plans share: the handle, the device, and the checks of tensors."""

    _name = ""

    def _open(self, desc, f16: bool) -> None:
        import torch

        self._lib = _library()
        self._h = None
        h = ctypes.c_void_p()
        _check(getattr(self._lib, f"agmm_{self._name}_plan")(ctypes.byref(desc), ctypes.byref(h)))
        self._h = h
        self._run = getattr(self._lib, f"agmm_{self._name}_run")
        self.dtype = torch.float16 if f16 else torch.bfloat16
        self.device = torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index
        self._current_stream = torch._C._cuda_getCurrentRawStream
        self._int32, self._int64 = torch.int32, torch.int64

    def close(self) -> None:
        if getattr(self, "_h", None):
            getattr(self._lib, f"agmm_{self._name}_destroy")(self._h)
            self._h = None

    def __del__(self):  # pragma: no cover
        try:
            self.close()
        except Exception:
            pass

    def _heads(self, name, x, heads):
        """(pointer, token stride, head stride) of a [rows, heads, head_dim] tensor."""
        shape, stride = x.shape, x.stride()
        if len(shape) != 3 or shape[1] != heads or shape[2] != self.head_dim or stride[2] != 1:
            raise ValueError(f"{name} must be [rows, {heads}, {self.head_dim}] with a contiguous last dimension, "
                             f"got {tuple(shape)} with strides {stride}")
        if x.dtype != self.dtype or x.device != self.device:
            raise ValueError(f"{name} must be {self.dtype} on {self.device}, got {x.dtype} on {x.device}")
        return x.data_ptr(), stride[0], stride[1]

    def _vector(self, name, x, dtype, size):
        """Pointer of a contiguous vector of `size` values."""
        if x.dtype != dtype or x.device != self.device or x.shape != (size,) or not x.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} vector of {size} on {self.device}, "
                             f"got {x.dtype} {tuple(x.shape)} on {x.device}")
        return x.data_ptr()

    def _caches(self, k_cache, v_cache, page_size=None):
        """(k pointer, v pointer, shape, strides) of two [pages, page_size, kv_heads, head_dim] tensors laid out alike."""
        shape, stride = k_cache.shape, k_cache.stride()
        if (len(shape) != 4 or shape[2] != self.kv_heads or shape[3] != self.head_dim or stride[3] != 1
                or (page_size is not None and shape[1] != page_size)):
            raise ValueError(f"k_cache must be [pages, {page_size or 'page_size'}, {self.kv_heads}, {self.head_dim}] with a "
                             f"contiguous last dimension, got {tuple(shape)} with strides {stride}")
        if v_cache.shape != shape or v_cache.stride() != stride:
            raise ValueError("k_cache and v_cache must share one shape and strides")
        for x in (k_cache, v_cache):
            if x.dtype != self.dtype or x.device != self.device:
                raise ValueError(f"the caches must be {self.dtype} on {self.device}, got {x.dtype} on {x.device}")
        return k_cache.data_ptr(), v_cache.data_ptr(), shape, stride

    def _stream(self, stream):
        if stream is None:
            return self._current_stream(self._index)
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)

    def workspace_bytes(self) -> int:
        return int(getattr(self._lib, f"agmm_{self._name}_workspace_bytes")(self._h))

    def new_workspace(self):
        """A zero-filled workspace.  It is zeroed on the current stream: runs on
        another stream must first wait for it."""
        import torch

        return torch.zeros(self.workspace_bytes(), dtype=torch.uint8, device=self.device)

    def _workspace(self, workspace):
        if workspace.device != self.device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous on {self.device}")
        if workspace.numel() * workspace.element_size() < self._workspace_size:
            raise ValueError(f"workspace needs {self._workspace_size} bytes")
        return workspace.data_ptr()

    def query_status(self, workspace, stream=None) -> int:
        """Synchronize and return (and clear) the device status; raises on error.
        The workspace can be used again after that."""
        st = self._lib.agmm_query_status(None, workspace.data_ptr(), self._stream(stream))
        _check(st)
        return st


def rotary_axes(sections: Sequence[int], interleaved: bool = False) -> List[int]:
    """The position axis of each rotary pair.  ``sections`` counts the pairs of
    each axis; contiguous runs, or (interleaved) dealt out in turn until an
    axis has all of its pairs."""
    if not interleaved:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                out.append(a)
                left[a] -= 1
    return out


class NormRopePlan(_AttentionPlan):
    """RMS norm of query and key heads and their rotation by position, into
    packed rows and cache slots (agmm_norm_rope_run).

    sections: pairs of each position axis (default: one axis); their sum is
    rotary_dim / 2.  interleaved: see rotary_axes.  adjacent: pairs are (2i,
    2i + 1) rather than (i, i + rotary_dim / 2).  inv_freq: the pairs'
    frequencies in radians per position (default: base^(-2i / rotary_dim))."""

    _name = "norm_rope"

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, rotary_dim: Optional[int] = None,
                 sections: Optional[Sequence[int]] = None, interleaved: bool = False, adjacent: bool = False,
                 base: float = 10000.0, inv_freq: Optional[Sequence[float]] = None, eps: float = 1e-6,
                 f16: bool = False):
        self.q_heads, self.kv_heads, self.head_dim = int(q_heads), int(kv_heads), int(head_dim)
        self.rotary_dim = self.head_dim if rotary_dim is None else int(rotary_dim)
        pairs = self.rotary_dim // 2
        sections = (pairs,) if sections is None else tuple(int(n) for n in sections)
        if sum(sections) != pairs or any(n < 0 for n in sections):
            raise ValueError(f"sections must sum to rotary_dim / 2 = {pairs}, got {sections}")
        if inv_freq is None:
            inv_freq = [float(base) ** (-2.0 * i / self.rotary_dim) for i in range(pairs)]
        inv_freq = [float(f) for f in inv_freq]
        if len(inv_freq) != pairs:
            raise ValueError(f"inv_freq must have rotary_dim / 2 = {pairs} values, got {len(inv_freq)}")
        self.axes = len(sections)
        self.adjacent = bool(adjacent)
        freq = (ctypes.c_double * max(1, pairs))(*inv_freq)
        axis = (ctypes.c_int * max(1, pairs))(*rotary_axes(sections, interleaved))
        desc = _NormRopeDesc(self.q_heads, self.kv_heads, self.head_dim, self.rotary_dim, int(self.adjacent), self.axes,
                             AGMM_F16 if f16 else AGMM_BF16, float(eps), freq, axis)
        self._open(desc, f16)

    def run(self, qkv, q_weight, k_weight, positions, q, k=None, k_cache=None, v_cache=None, slots=None,
            stream=None) -> None:
        """qkv [tokens, (q_heads + 2 kv_heads) * head_dim] (or with heads as a
        dimension of their own), q_weight and k_weight [head_dim] (both None:
        no norm), positions [axes, tokens] or, with one axis, [tokens], int32 or
        int64.  Outputs: q and k [tokens, heads, head_dim] (either may be qkv's
        own part), and k_cache, v_cache [pages, page_size, kv_heads, head_dim] at
        slots [tokens] int64 (page * page_size + place; one outside the cache,
        as -1, is not written)."""
        shape, stride, d = qkv.shape, qkv.stride(), self.head_dim
        heads = self.q_heads + 2 * self.kv_heads
        if len(shape) == 2 and shape[1] == heads * d and stride[1] == 1:
            qkv_ptr, qkv_ts, qkv_hs = qkv.data_ptr(), stride[0], d
            if qkv.dtype != self.dtype or qkv.device != self.device:
                raise ValueError(f"qkv must be {self.dtype} on {self.device}, got {qkv.dtype} on {qkv.device}")
        else:
            qkv_ptr, qkv_ts, qkv_hs = self._heads("qkv", qkv, heads)
        tokens = shape[0]
        q_ptr, q_ts, q_hs = self._heads("q", q, self.q_heads)
        if q.shape[0] != tokens:
            raise ValueError(f"q must have {tokens} rows, got {q.shape[0]}")
        k_ptr = k_ts = k_hs = 0
        if k is not None:
            k_ptr, k_ts, k_hs = self._heads("k", k, self.kv_heads)
            if k.shape[0] != tokens:
                raise ValueError(f"k must have {tokens} rows, got {k.shape[0]}")
        qw = kw = 0
        if q_weight is not None or k_weight is not None:
            if q_weight is None or k_weight is None:
                raise ValueError("q_weight and k_weight are given together or not at all")
            qw = self._vector("q_weight", q_weight, self.dtype, d)
            kw = self._vector("k_weight", k_weight, self.dtype, d)
        pos_ptr = pos_bytes = pos_stride = 0
        if self.rotary_dim:
            ps = positions.shape
            if not (ps == (self.axes, tokens) or (self.axes == 1 and ps == (tokens,))) or positions.device != self.device \
                    or positions.dtype not in (self._int32, self._int64) or (tokens > 1 and positions.stride(-1) != 1):
                raise ValueError(f"positions must be int32 or int64 [{self.axes}, {tokens}] on {self.device} with contiguous rows, "
                                 f"got {positions.dtype} {tuple(ps)} on {positions.device}")
            pos_ptr, pos_bytes = positions.data_ptr(), 8 if positions.dtype == self._int64 else 4
            pos_stride = positions.stride(0) if len(ps) == 2 else 0
        kc = vc = pages = page = c_ps = c_ts = c_hs = slot_ptr = 0
        if k_cache is not None or v_cache is not None:
            if k_cache is None or v_cache is None or slots is None:
                raise ValueError("k_cache, v_cache and slots are given together or not at all")
            kc, vc, (pages, page, _, _), (c_ps, c_ts, c_hs, _) = self._caches(k_cache, v_cache)
            slot_ptr = self._vector("slots", slots, self._int64, tokens)
        args = _NORM_ROPE_ARGS.pack(tokens, qkv_ptr, qkv_ts, qkv_hs, qw, kw, pos_ptr, pos_bytes, pos_stride, q_ptr, q_ts, q_hs,
                                    k_ptr, k_ts, k_hs, kc, vc, pages, page, c_ps, c_ts, c_hs, slot_ptr)
        st = self._run(self._h, args, self._stream(stream))
        if st:
            _check(st)


class PromptPlan(_AttentionPlan):
    """Attention of packed prompts with grouped heads (agmm_prompt_run)."""

    _name = "prompt"

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, scale: Optional[float] = None, causal: bool = True,
                 f16: bool = False):
        self.q_heads, self.kv_heads, self.head_dim = int(q_heads), int(kv_heads), int(head_dim)
        self.scale = self.head_dim ** -0.5 if scale is None else float(scale)
        self.causal = bool(causal)
        self._open(_PromptDesc(self.q_heads, self.kv_heads, self.head_dim, int(self.causal),
                               AGMM_F16 if f16 else AGMM_BF16, self.scale), f16)
        self._workspace_size = self.workspace_bytes()

    def run(self, q, k, v, starts, out, workspace, kv_starts=None, stream=None) -> None:
        """q [tokens, q_heads, head_dim], k and v [kv_tokens, kv_heads,
        head_dim], starts [sequences + 1] int32: the rows of q where each
        sequence starts, and the end.  kv_starts: the same of k and v, when
        they are not starts; a sequence with more keys than queries has its
        queries at its end."""
        hk = self.kv_heads
        q_ptr, q_ts, q_hs = self._heads("q", q, self.q_heads)
        k_ptr, k_ts, k_hs = self._heads("k", k, hk)
        v_ptr, v_ts, v_hs = self._heads("v", v, hk)
        o_ptr, o_ts, o_hs = self._heads("out", out, self.q_heads)
        tokens, kv_tokens = q.shape[0], k.shape[0]
        if out.shape[0] != tokens or v.shape[0] != kv_tokens:
            raise ValueError(f"out must have q's {tokens} rows and v k's {kv_tokens}, got {out.shape[0]} and {v.shape[0]}")
        edges = starts.shape[0] if starts.dim() == 1 else 0
        if edges < 1:
            raise ValueError("starts must be a vector of sequences + 1 values")
        s_ptr = self._vector("starts", starts, self._int32, edges)
        if kv_starts is None:
            ks_ptr = 0
            if kv_tokens != tokens:
                raise ValueError(f"q has {tokens} rows and k {kv_tokens}: give kv_starts")
        else:
            ks_ptr = self._vector("kv_starts", kv_starts, self._int32, edges)
        args = _PROMPT_ARGS.pack(tokens, kv_tokens, edges - 1, q_ptr, q_ts, q_hs, k_ptr, k_ts, k_hs, v_ptr, v_ts, v_hs,
                                 o_ptr, o_ts, o_hs, s_ptr, ks_ptr, self._workspace(workspace))
        st = self._run(self._h, args, self._stream(stream))
        if st:
            _check(st)


class TreePlan(_AttentionPlan):
    """Attention of drafted tokens, or of single ones, over a paged cache
    (agmm_tree_run).  max_nodes: the most drafted tokens of a sequence."""

    _name = "tree"

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, page_size: int, max_nodes: int = 1,
                 scale: Optional[float] = None, f16: bool = False):
        self.q_heads, self.kv_heads, self.head_dim = int(q_heads), int(kv_heads), int(head_dim)
        self.page_size, self.max_nodes = int(page_size), int(max_nodes)
        self.scale = self.head_dim ** -0.5 if scale is None else float(scale)
        self._open(_TreeDesc(self.q_heads, self.kv_heads, self.head_dim, self.page_size, self.max_nodes,
                             AGMM_F16 if f16 else AGMM_BF16, self.scale), f16)
        self._workspace_size = self.workspace_bytes()

    def run(self, q, k_cache, v_cache, page_table, context_lens, node_starts, out, workspace, mask=None,
            stream=None) -> None:
        """q [tokens, q_heads, head_dim], the drafted tokens of all sequences;
        k_cache, v_cache [pages, page_size, kv_heads, head_dim], which hold each
        sequence's context and, after it, its drafted tokens; page_table
        [sequences, pages of one] int32; context_lens [sequences] int32;
        node_starts [sequences + 1] int32; mask [tokens, words] int64, see
        tree_mask (None: each drafted token sees those before it)."""
        q_ptr, q_ts, q_hs = self._heads("q", q, self.q_heads)
        o_ptr, o_ts, o_hs = self._heads("out", out, self.q_heads)
        kc, vc, shape, (c_ps, c_ts, c_hs, _) = self._caches(k_cache, v_cache, self.page_size)
        tokens = q.shape[0]
        if out.shape[0] != tokens:
            raise ValueError(f"out must have q's {tokens} rows, got {out.shape[0]}")
        table = page_table.shape
        if len(table) != 2 or page_table.dtype != self._int32 or page_table.device != self.device or page_table.stride(1) != 1:
            raise ValueError(f"page_table must be int32 [sequences, pages] on {self.device} with contiguous rows")
        sequences = table[0]
        c_ptr = self._vector("context_lens", context_lens, self._int32, sequences)
        n_ptr = self._vector("node_starts", node_starts, self._int32, sequences + 1)
        m_ptr = words = 0
        if mask is not None:
            if mask.dim() != 2 or mask.shape[0] != tokens or mask.dtype != self._int64 or mask.device != self.device \
                    or not mask.is_contiguous():
                raise ValueError(f"mask must be contiguous int64 [{tokens}, words] on {self.device}")
            m_ptr, words = mask.data_ptr(), mask.shape[1]
        args = _TREE_ARGS.pack(tokens, sequences, q_ptr, q_ts, q_hs, kc, vc, shape[0], c_ps, c_ts, c_hs,
                               page_table.data_ptr(), table[1], page_table.stride(0), c_ptr, n_ptr, m_ptr, words, o_ptr, o_ts, o_hs,
                               self._workspace(workspace))
        st = self._run(self._h, args, self._stream(stream))
        if st:
            _check(st)


def tree_mask(parents: Sequence[Sequence[int]], words: Optional[int] = None, device=None):
    """The mask of TreePlan.run for trees given by their nodes' parents:
    parents[s][i] < i is the parent of node i of sequence s, -1 at a root.
    Every node sees itself and its ancestors."""
    import torch

    most = max([len(p) for p in parents], default=0)
    need = max(1, (most + 63) // 64)
    words = need if words is None else int(words)
    if words < need:
        raise ValueError(f"{most} nodes need {need} words, got {words}")
    out = []
    for tree in parents:
        rows: List[int] = []
        for i, p in enumerate(tree):
            if not -1 <= p < i:
                raise ValueError(f"the parent of node {i} must be in [-1, {i - 1}]: {p}")
            rows.append((rows[p] if p >= 0 else 0) | 1 << i)
        for r in rows:
            at = [(r >> 64 * w) & (1 << 64) - 1 for w in range(words)]
            out.append([v - (1 << 64) if v >> 63 else v for v in at])
    return torch.tensor(out, dtype=torch.int64, device=device or "cuda").view(-1, words)


_plans: Dict[tuple, _AttentionPlan] = {}


def _cached(cls, *args, **kw):
    import torch

    key = (cls, args, tuple(sorted(kw.items())), torch.cuda.current_device())
    plan = _plans.get(key)
    if plan is None:
        plan = _plans[key] = cls(*args, **kw)
    return plan


def _is_f16(x) -> bool:
    import torch

    if x.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("inputs must be bfloat16 or float16")
    return x.dtype == torch.float16


def qkv_norm_rope(qkv, q_weight, k_weight, positions, q_heads: int, kv_heads: int, k_cache=None, v_cache=None, slots=None,
                  rotary_dim: Optional[int] = None, sections: Optional[Sequence[int]] = None, interleaved: bool = False,
                  adjacent: bool = False, base: float = 10000.0, eps: float = 1e-6, stream=None):
    """Norms and rotates the heads of a QKV product [tokens, (q_heads + 2
    kv_heads) * head_dim]; returns (q, k), each [tokens, heads, head_dim], and
    writes keys and values to the caches when they are given (NormRopePlan)."""
    import torch

    heads = int(q_heads) + 2 * int(kv_heads)
    if qkv.dim() != 2 or qkv.shape[1] % heads:
        raise ValueError(f"qkv must be [tokens, {heads} * head_dim], got {tuple(qkv.shape)}")
    d = qkv.shape[1] // heads
    plan = _cached(NormRopePlan, int(q_heads), int(kv_heads), d, rotary_dim=rotary_dim,
                   sections=None if sections is None else tuple(sections), interleaved=bool(interleaved),
                   adjacent=bool(adjacent), base=float(base), eps=float(eps), f16=_is_f16(qkv))
    with _On(stream):
        q = torch.empty((qkv.shape[0], q_heads, d), dtype=qkv.dtype, device=qkv.device)
        k = torch.empty((qkv.shape[0], kv_heads, d), dtype=qkv.dtype, device=qkv.device)
    plan.run(qkv, q_weight, k_weight, positions, q, k=k, k_cache=k_cache, v_cache=v_cache, slots=slots, stream=stream)
    return q, k


def prompt_attention(q, k, v, starts, kv_starts=None, scale: Optional[float] = None, causal: bool = True, out=None,
                     workspace=None, stream=None):
    """Attention of packed prompts; returns [tokens, q_heads, head_dim] (PromptPlan)."""
    import torch

    plan = _cached(PromptPlan, q.shape[1], k.shape[1], q.shape[2], scale=scale, causal=bool(causal), f16=_is_f16(q))
    with _On(stream):
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if workspace is None:
            workspace = plan.new_workspace()
    plan.run(q, k, v, starts, out, workspace, kv_starts=kv_starts, stream=stream)
    return out


def tree_attention(q, k_cache, v_cache, page_table, context_lens, node_starts, mask=None, max_nodes: Optional[int] = None,
                   scale: Optional[float] = None, out=None, workspace=None, stream=None):
    """Attention of drafted tokens over a paged cache; returns [tokens,
    q_heads, head_dim] (TreePlan).

    max_nodes: the most drafted tokens of a sequence, 1 for the ordinary decode
    step.  It is not known on the host; without it room is made for all of q's
    tokens in one sequence (1024 of them at most), and a workspace as large is
    zeroed: give it where the time of a call counts.  Rows past it are zero in an
    output that is made here, as it is the plan that bounds them."""
    import torch

    tokens, sequences = q.shape[0], page_table.shape[0]
    bound = max_nodes
    if max_nodes is None:
        # a power of two: few plans for all numbers of tokens
        max_nodes = min(MAX_NODES, 1 << max(0, tokens - 1).bit_length())
        if mask is not None and mask.dim() == 2 and mask.shape[1] < (max_nodes + 63) // 64:
            with _On(stream):  # words that are not there have no bit set
                mask = torch.nn.functional.pad(mask, (0, (max_nodes + 63) // 64 - mask.shape[1]))
    elif tokens > sequences * int(max_nodes):
        raise ValueError(f"{tokens} drafted tokens of {sequences} sequences: some have more than max_nodes = {max_nodes}")
    plan = _cached(TreePlan, q.shape[1], k_cache.shape[2], q.shape[2], page_size=k_cache.shape[1], max_nodes=int(max_nodes),
                   scale=scale, f16=_is_f16(q))
    with _On(stream):
        if out is None:
            # zeros where a sequence could have rows past the bound
            out = (torch.zeros if tokens > plan.max_nodes else torch.empty)(q.shape, dtype=q.dtype, device=q.device)
        if workspace is None:
            workspace = plan.new_workspace()
        elif bound is None and workspace.numel() * workspace.element_size() < plan.workspace_bytes():
            raise ValueError(f"without max_nodes, room is made for {plan.max_nodes} drafted tokens to a sequence, which needs a "
                             f"workspace of {plan.workspace_bytes()} bytes: give the max_nodes that this one was made for")
    plan.run(q, k_cache, v_cache, page_table, context_lens, node_starts, out, workspace, mask=mask, stream=stream)
    return out
