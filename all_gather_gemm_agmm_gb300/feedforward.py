"""The feed-forward half of a transformer block around the gathered product:
layer norm, the gated product, and the product with bias, activation and
residual, each with its backward pass.

Every step of the computation runs in the CUDA kernels of ``libagmm.so``
(``include/agmm_feedforward.h``, which defines each operator); this module
checks arguments and marshals them.  PyTorch supplies device memory and
streams.  There is no CPU fallback.

As with :class:`Plan`, a plan is made once for a layer's shape, and its ``run``
and ``backward`` take the caller's buffers; the functions ``layer_norm``,
``gated_matmul`` and ``linear_matmul`` and their ``*_backward`` allocate them.
X comes as the shards of a gathered product (a list of [rows, k] tensors) or as
one tensor.  Nothing is recorded for PyTorch's autograd: a tensor that requires
grad is refused while grad mode is on (wrap the calls in a
``torch.autograd.Function``, whose forward and backward run without it).
Buffers follow PyTorch's stream rules: a tensor used on a ``stream`` other than
the one it was made on has to be ready there, and to outlive the work.  A
``stream`` is a ``torch.cuda.Stream``, an object with a ``cuda_stream`` handle, or
the handle; what the functions allocate belongs to it.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

from . import AGMM_BF16, AGMM_F16, _check, _On, load_library
from .attention import _AttentionPlan, _cached, _is_f16

FEEDFORWARD_SYMBOLS = [f"agmm_{op}_{f}" for op in ("layer_norm", "gated", "linear")
                       for f in ("plan", "workspace_bytes", "run", "backward", "destroy")]
FEEDFORWARD_SYMBOLS += ["agmm_gated_save_float", "agmm_linear_save_float"]
MAX_SHARDS = 8
HEAD_BYTES = 65536  # of a workspace: zero before its first use
ACTIVATIONS = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


class _LayerNormDesc(ctypes.Structure):
    _fields_ = [("columns", ctypes.c_int), ("dtype", ctypes.c_int), ("eps", ctypes.c_float)]


class _ProductDesc(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in ("k", "n", "activation", "rhs_transpose", "dtype")]


# The argument structs are 64-bit fields throughout.
_LAYER_NORM_ARGS = struct.Struct("9q")
_LAYER_NORM_GRAD_ARGS = struct.Struct("16q")
_GATED_ARGS = struct.Struct("20q")
_GATED_GRAD_ARGS = struct.Struct("29q")
_LINEAR_ARGS = struct.Struct("21q")
_LINEAR_GRAD_ARGS = struct.Struct("26q")

_bound = None


def _library():
    """libagmm.so with the signatures of agmm_feedforward.h declared."""
    global _bound
    if _bound is not None:
        return _bound
    lib = load_library()
    vp, c_int, out = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(ctypes.c_void_p)
    for name, desc in (("layer_norm", _LayerNormDesc), ("gated", _ProductDesc), ("linear", _ProductDesc)):
        f = getattr(lib, f"agmm_{name}_plan")
        f.argtypes, f.restype = [ctypes.POINTER(desc), out], c_int
        for call in ("run", "backward"):
            f = getattr(lib, f"agmm_{name}_{call}")
            f.argtypes, f.restype = [vp, ctypes.c_char_p, vp], c_int
        if name != "layer_norm":
            f = getattr(lib, f"agmm_{name}_save_float")
            f.argtypes, f.restype = [vp, c_int], c_int
        f = getattr(lib, f"agmm_{name}_workspace_bytes")
        f.argtypes, f.restype = [vp], ctypes.c_size_t
        f = getattr(lib, f"agmm_{name}_destroy")
        f.argtypes, f.restype = [vp], None
    _bound = lib
    return lib


class _FeedForwardPlan(_AttentionPlan):
    """What the three plans share: the handle, the device, and the checks of tensors."""

    def _open(self, desc, f16: bool) -> None:
        import torch

        _library()
        super()._open(desc, f16)
        self._backward = getattr(self._lib, f"agmm_{self._name}_backward")
        self._float32 = torch.float32
        self._grad_mode = torch.is_grad_enabled
        self._workspace_size = self.workspace_bytes()

    def new_workspace(self):
        """A workspace whose head is zero-filled.  It is zeroed on the current
        stream: runs on another stream must first wait for it."""
        import torch

        ws = torch.empty(self._workspace_size, dtype=torch.uint8, device=self.device)
        ws[:HEAD_BYTES].zero_()
        return ws

    def query_status(self, workspace, stream=None) -> int:
        """Synchronize and return (and clear) the device status; raises on error,
        with the workspace's head zero-filled for its next use."""
        import torch

        try:
            return super().query_status(workspace, stream)
        except Exception:
            with _On(stream):
                workspace.view(-1).view(torch.uint8)[:HEAD_BYTES].zero_()
            raise

    def _matrix(self, name, x, rows, cols, dtype=None):
        """(pointer, row stride) of a [rows, cols] tensor."""
        stride = x.stride()
        if x.shape != (rows, cols) or stride[1] != 1:
            raise ValueError(f"{name} must be [{rows}, {cols}] with a contiguous last dimension, "
                             f"got {tuple(x.shape)} with strides {stride}")
        if x.dtype is not (dtype or self.dtype) or x.get_device() != self._index or x.requires_grad:
            self._check(name, x, dtype)
        return x.data_ptr(), stride[0]

    def _check(self, name, x, dtype):
        if x.dtype is not (dtype or self.dtype) or x.get_device() != self._index:
            raise ValueError(f"{name} must be {dtype or self.dtype} on {self.device}, got {x.dtype} on {x.device}")
        if x.requires_grad and self._grad_mode():
            raise ValueError(f"{name} requires grad, and nothing is recorded here: call under torch.no_grad()")

    def _workspace(self, workspace):
        if workspace.get_device() != self._index or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous on {self.device}")
        if workspace.nbytes < self._workspace_size:
            raise ValueError(f"workspace needs {self._workspace_size} bytes")
        return workspace.data_ptr()

    def _pair(self, names, xs, rows, cols, dtype=None):
        """(pointer, pointer, row stride) of two [rows, cols] tensors laid out alike."""
        a, sa = self._matrix(names[0], xs[0], rows, cols, dtype)
        b, sb = self._matrix(names[1], xs[1], rows, cols, dtype)
        if sa != sb and rows > 1:
            raise ValueError(f"{names[0]} and {names[1]} must share one row stride, got {sa} and {sb}")
        return a, b, sa

    def _values(self, name, x, size, dtype=None):
        """Pointer of a contiguous vector of `size` values; 0 for None."""
        if x is None:
            return 0
        if x.shape != (size,) or not x.is_contiguous():
            raise ValueError(f"{name} must be a contiguous vector of {size}, got {tuple(x.shape)} with strides {x.stride()}")
        if x.dtype is not (dtype or self.dtype) or x.get_device() != self._index or x.requires_grad:
            self._check(name, x, dtype)
        return x.data_ptr()

    def _grad_type(self, a, b):
        """The type of the weights' gradients: the plan's, or float32 for all of them."""
        f32 = self._float32
        if a is None:
            return f32 if b is not None and b.dtype is f32 else self.dtype
        if b is not None and (a.dtype is f32) != (b.dtype is f32):
            raise ValueError(f"the gradients of the weights must all be {self.dtype} or all float32, got {a.dtype} and {b.dtype}")
        return f32 if a.dtype is f32 else self.dtype

    def _call(self, f, args, stream):
        st = f(self._h, args, self._stream(stream))
        if st:
            _check(st)


def _width(name, v):
    v = int(v)
    if not -2**31 <= v < 2**31:  # an int of the plan's description
        raise ValueError(f"{name} must be a 32-bit number, got {v}")
    return v


class LayerNormPlan(_FeedForwardPlan):
    """Layer norm of rows and its backward pass (agmm_layer_norm_run, _backward)."""

    _name = "layer_norm"

    def __init__(self, columns: int, eps: float = 1e-5, f16: bool = False):
        self.columns, self.eps = _width("columns", columns), float(eps)
        self._open(_LayerNormDesc(self.columns, AGMM_F16 if f16 else AGMM_BF16, self.eps), f16)

    def run(self, x, out, weight=None, bias=None, mean=None, rstd=None, stream=None) -> None:
        """x and out [rows, columns] (out may be x), weight and bias [columns].
        mean and rstd [rows] float32: written for the backward pass."""
        c, rows = self.columns, x.shape[0]
        x_ptr, x_s = self._matrix("x", x, rows, c)
        o_ptr, o_s = self._matrix("out", out, rows, c)
        args = _LAYER_NORM_ARGS.pack(rows, x_ptr, x_s, self._values("weight", weight, c), self._values("bias", bias, c), o_ptr, o_s,
                                     self._values("mean", mean, rows, self._float32), self._values("rstd", rstd, rows, self._float32))
        self._call(self._run, args, stream)

    def backward(self, d_out, x, mean, rstd, dx, workspace, weight=None, add=None, d_weight=None, d_bias=None, stream=None) -> None:
        """d_out, x [rows, columns], mean and rstd [rows] as the forward pass wrote
        them, weight as it was there.  Outputs, each of them optional: dx [rows,
        columns] (None: not wanted; it may be d_out or add; add is added to it),
        d_weight and d_bias [columns], both of the plan's type or both float32.
        workspace may be None without those two."""
        c, rows = self.columns, x.shape[0]
        d_ptr, d_s = self._matrix("d_out", d_out, rows, c)
        x_ptr, x_s = self._matrix("x", x, rows, c)
        a_ptr, a_s = (0, 0) if add is None else self._matrix("add", add, rows, c)
        dx_ptr, dx_s = (0, 0) if dx is None else self._matrix("dx", dx, rows, c)
        grads = self._grad_type(d_weight, d_bias)
        if workspace is None and d_weight is None and d_bias is None:
            ws = 0
        else:
            ws = self._workspace(workspace)
        args = _LAYER_NORM_GRAD_ARGS.pack(rows, d_ptr, d_s, x_ptr, x_s, self._values("mean", mean, rows, self._float32),
                                          self._values("rstd", rstd, rows, self._float32), self._values("weight", weight, c), a_ptr,
                                          a_s, dx_ptr, dx_s, self._values("d_weight", d_weight, c, grads),
                                          self._values("d_bias", d_bias, c, grads), grads is self._float32, ws)
        self._call(self._backward, args, stream)


class _ProductPlan(_FeedForwardPlan):
    def __init__(self, k: int, n: int, activation: Optional[str], rhs_transpose: bool, f16: bool, f32_saved: bool):
        if activation not in ACTIVATIONS:
            raise ValueError(f"activation must be one of {list(ACTIVATIONS)}, got {activation!r}")
        self.k, self.n, self.activation, self.rhs_transpose = _width("k", k), _width("n", n), activation, bool(rhs_transpose)
        self._weight_shape = (self.n, self.k) if self.rhs_transpose else (self.k, self.n)
        self._open(_ProductDesc(self.k, self.n, ACTIVATIONS[activation], int(self.rhs_transpose), AGMM_F16 if f16 else AGMM_BF16), f16)
        self.f32_saved = bool(f32_saved)
        self._saved = self._float32 if self.f32_saved else self.dtype  # the type of what the forward pass saves
        if self.f32_saved:
            _check(getattr(self._lib, f"agmm_{self._name}_save_float")(self._h, 1))

    def _shards(self, xs):
        """(shards, rows, 8 pointers, row stride) of X."""
        if not isinstance(xs, (list, tuple)):
            xs = (xs,)
        if not 1 <= len(xs) <= MAX_SHARDS:
            raise ValueError(f"X must be 1 to {MAX_SHARDS} shards, got {len(xs)}")
        rows = xs[0].shape[0]
        ptrs, stride = [0] * MAX_SHARDS, 0
        for i, x in enumerate(xs):
            ptrs[i], s = self._matrix("a shard of X", x, rows, self.k)
            if i and rows > 1 and s != stride:
                raise ValueError(f"the shards of X must share one row stride, got {stride} and {s}")
            stride = s
        return len(xs), rows, ptrs, stride


class GatedPlan(_ProductPlan):
    """The gated product act(X Wgate) * (X Wup) in one kernel, and its backward
    pass (agmm_gated_run, _backward).  Weights [k, n], or [n, k] with
    rhs_transpose; activation: "silu", "gelu", "gelu_tanh" or "relu".  f32_saved:
    gate and up are float32, for gradients without their rounding."""

    _name = "gated"

    def __init__(self, k: int, n: int, activation: str = "silu", rhs_transpose: bool = False, f16: bool = False,
                 f32_saved: bool = False):
        super().__init__(k, n, activation, rhs_transpose, f16, f32_saved)

    def run(self, xs, w_gate, w_up, out, workspace, gate=None, up=None, stream=None) -> None:
        """xs: [rows, k], or up to 8 such shards; out [tokens, n].  gate and up
        [tokens, n]: written for the backward pass.  The two weights (and gate and
        up) may be halves of one tensor."""
        shards, rows, xp, x_s = self._shards(xs)
        tokens = shards * rows
        wg, wu, w_s = self._pair(("w_gate", "w_up"), (w_gate, w_up), *self._weight_shape)
        o_ptr, o_s = self._matrix("out", out, tokens, self.n)
        g = u = s_s = 0
        if gate is not None or up is not None:
            if gate is None or up is None:
                raise ValueError("gate and up are given together or not at all")
            g, u, s_s = self._pair(("gate", "up"), (gate, up), tokens, self.n, self._saved)
        args = _GATED_ARGS.pack(shards, rows, *xp, x_s, wg, wu, w_s, o_ptr, o_s, g, u, s_s, self._workspace(workspace))
        self._call(self._run, args, stream)

    def backward(self, d_out, xs, w_gate, w_up, gate, up, d_gate, d_up, workspace, dx=None, dw_gate=None, dw_up=None,
                 stream=None) -> None:
        """d_out [tokens, n]; xs and the weights as the forward pass had them, gate
        and up as it wrote them.  d_gate and d_up [tokens, n]: written on the way
        (they may be gate and up, unless those are float32).  Outputs: dx [tokens, k], and dw_gate and dw_up
        like the weights, of the plan's type or float32; what is None is not computed."""
        shards, rows, xp, x_s = self._shards(xs)
        tokens = shards * rows
        wg, wu, w_s = self._pair(("w_gate", "w_up"), (w_gate, w_up), *self._weight_shape)
        o_ptr, o_s = self._matrix("d_out", d_out, tokens, self.n)
        g, u, s_s = self._pair(("gate", "up"), (gate, up), tokens, self.n, self._saved)
        dg, du, d_s = self._pair(("d_gate", "d_up"), (d_gate, d_up), tokens, self.n)
        dx_ptr, dx_s = (0, 0) if dx is None else self._matrix("dx", dx, tokens, self.k)
        grads = self._grad_type(dw_gate, dw_up)
        dwg = dwu = dw_s = 0
        if dw_gate is not None or dw_up is not None:
            if dw_gate is None or dw_up is None:
                raise ValueError("dw_gate and dw_up are given together or not at all")
            dwg, dwu, dw_s = self._pair(("dw_gate", "dw_up"), (dw_gate, dw_up), *self._weight_shape, grads)
        args = _GATED_GRAD_ARGS.pack(shards, rows, *xp, x_s, wg, wu, w_s, o_ptr, o_s, g, u, s_s, dg, du, d_s, dx_ptr, dx_s, dwg, dwu,
                                     dw_s, grads is self._float32, self._workspace(workspace))
        self._call(self._backward, args, stream)


class LinearPlan(_ProductPlan):
    """The product act(X W + bias) + residual in one kernel, and its backward pass
    (agmm_linear_run, _backward).  The weight [k, n], or [n, k] with rhs_transpose;
    activation: None, "silu", "gelu", "gelu_tanh" or "relu".  f32_saved: pre is
    float32, for gradients without its rounding."""

    _name = "linear"

    def __init__(self, k: int, n: int, activation: Optional[str] = None, rhs_transpose: bool = False, f16: bool = False,
                 f32_saved: bool = False):
        super().__init__(k, n, activation, rhs_transpose, f16, f32_saved)

    def run(self, xs, w, out, workspace, bias=None, residual=None, pre=None, stream=None) -> None:
        """xs: [rows, k], or up to 8 such shards; bias [n]; residual and out
        [tokens, n] (out may be residual).  pre [tokens, n]: X W + bias, written
        for the backward pass."""
        shards, rows, xp, x_s = self._shards(xs)
        tokens = shards * rows
        w_ptr, w_s = self._matrix("w", w, *self._weight_shape)
        r_ptr, r_s = (0, 0) if residual is None else self._matrix("residual", residual, tokens, self.n)
        o_ptr, o_s = self._matrix("out", out, tokens, self.n)
        p_ptr, p_s = (0, 0) if pre is None else self._matrix("pre", pre, tokens, self.n, self._saved)
        args = _LINEAR_ARGS.pack(shards, rows, *xp, x_s, w_ptr, w_s, self._values("bias", bias, self.n), r_ptr, r_s, o_ptr, o_s, p_ptr,
                                 p_s, self._workspace(workspace))
        self._call(self._run, args, stream)

    def backward(self, d_out, xs, w, workspace, pre=None, d_pre=None, dx=None, dw=None, d_bias=None, stream=None) -> None:
        """d_out [tokens, n]; xs and w as the forward pass had them.  With an
        activation: pre as the forward pass wrote it, and d_pre [tokens, n],
        written on the way (it may be d_out, or pre unless that is float32).  Outputs: dx [tokens, k], dw
        like the weight and d_bias [n], these two of the plan's type or both float32;
        what is None is not computed.  The residual's gradient is d_out."""
        shards, rows, xp, x_s = self._shards(xs)
        tokens = shards * rows
        w_ptr, w_s = self._matrix("w", w, *self._weight_shape)
        o_ptr, o_s = self._matrix("d_out", d_out, tokens, self.n)
        p_ptr, p_s = (0, 0) if pre is None else self._matrix("pre", pre, tokens, self.n, self._saved)
        d_ptr, d_s = (0, 0) if d_pre is None else self._matrix("d_pre", d_pre, tokens, self.n)
        dx_ptr, dx_s = (0, 0) if dx is None else self._matrix("dx", dx, tokens, self.k)
        grads = self._grad_type(dw, d_bias)
        dw_ptr, dw_s = (0, 0) if dw is None else self._matrix("dw", dw, *self._weight_shape, grads)
        args = _LINEAR_GRAD_ARGS.pack(shards, rows, *xp, x_s, w_ptr, w_s, o_ptr, o_s, p_ptr, p_s, d_ptr, d_s, dx_ptr, dx_s, dw_ptr,
                                      dw_s, self._values("d_bias", d_bias, self.n, grads), grads is self._float32,
                                      self._workspace(workspace))
        self._call(self._backward, args, stream)


# ------------------------------------------------------------------ the functions
def _rows(x):
    """x, or a copy of it where its rows do not lie as the kernels read them
    (a transposed or broadcast tensor, as a gradient may be)."""
    if x is None or x.dim() != 2:
        return x
    s = x.stride()
    if (s[1] == 1 or x.shape[1] == 1) and x.data_ptr() % 16 == 0 and (x.shape[0] <= 1 or (s[0] >= x.shape[1] and s[0] % 8 == 0)):
        return x
    return x.contiguous() if not x.is_contiguous() else x.clone()


def _vector(x):
    return x if x is None or (x.is_contiguous() and x.data_ptr() % 16 == 0) else x.clone(memory_format=_contiguous())


def _contiguous():
    import torch

    return torch.contiguous_format


def _list(xs):
    return list(xs) if isinstance(xs, (list, tuple)) else [xs]


def _shard_rows(xs):
    """The shards, each as the kernels read it, all with one row stride."""
    xs = [_rows(x) for x in xs]
    if len({x.stride(0) for x in xs}) > 1:
        xs = [x.contiguous() for x in xs]
    return xs


def _pair_rows(a, b):
    a, b = _rows(a), _rows(b)
    return (a, b) if a is None or b is None or a.stride(0) == b.stride(0) else (a.contiguous(), b.contiguous())


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, return_stats: bool = False, out=None, stream=None):
    """Layer norm of x [rows, columns]; returns the normed rows, with
    return_stats (rows, mean, rstd) as the backward pass reads them (LayerNormPlan)."""
    import torch

    if x.dim() != 2:
        raise ValueError(f"x must be [rows, columns], got {tuple(x.shape)}")
    plan = _cached(LayerNormPlan, x.shape[1], eps=float(eps), f16=_is_f16(x))
    mean = rstd = None
    with _On(stream):
        x, weight, bias = _rows(x), _vector(weight), _vector(bias)
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        if return_stats:
            mean, rstd = (torch.empty(x.shape[0], dtype=torch.float32, device=x.device) for _ in range(2))
    plan.run(x, out, weight=weight, bias=bias, mean=mean, rstd=rstd, stream=stream)
    return (out, mean, rstd) if return_stats else out


def layer_norm_backward(d_out, x, mean, rstd, weight=None, add=None, f32_grads: bool = False, workspace=None, stream=None):
    """(dx, d_weight, d_bias) of layer_norm; add is added to dx (the gradient that
    comes past the norm)."""
    import torch

    if x.dim() != 2:
        raise ValueError(f"x must be [rows, columns], got {tuple(x.shape)}")
    # the statistics have eps in them: any plan of these columns will do
    plan = _cached(LayerNormPlan, x.shape[1], eps=1e-5, f16=_is_f16(x))
    with _On(stream):
        d_out, x, add, weight = _rows(d_out), _rows(x), _rows(add), _vector(weight)
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        d_weight, d_bias = (torch.empty(x.shape[1], dtype=torch.float32 if f32_grads else x.dtype, device=x.device) for _ in range(2))
        if workspace is None:
            workspace = plan.new_workspace()
    plan.backward(d_out, x, mean, rstd, dx, workspace, weight=weight, add=add, d_weight=d_weight, d_bias=d_bias, stream=stream)
    return dx, d_weight, d_bias


def _product_sizes(xs, w, rhs_transpose):
    """The shards as a list, and (k, n)."""
    xs = _list(xs)
    if not xs or any(x.dim() != 2 for x in xs) or w.dim() != 2:
        raise ValueError("X must be [rows, k] or a list of such shards, and a weight a matrix")
    k, n = (w.shape[1], w.shape[0]) if rhs_transpose else tuple(w.shape)
    if xs[0].shape[1] != k:
        raise ValueError(f"contracting dimension mismatch: X has k={xs[0].shape[1]}, the weight gives {k}")
    return xs, k, n


def _product_plan(cls, k, n, activation, rhs_transpose, x, f32_saved):
    return _cached(cls, k, n, activation=activation, rhs_transpose=bool(rhs_transpose), f16=_is_f16(x), f32_saved=bool(f32_saved))


def gated_matmul(xs, w_gate, w_up, activation: str = "silu", rhs_transpose: bool = False, return_saved: bool = False, out=None,
                 workspace=None, stream=None, f32_saved: bool = False):
    """act(X Wgate) * (X Wup) of X [tokens, k] or the shards of a gathered X;
    returns [tokens, n], with return_saved (out, gate, up) as the backward pass
    reads them (GatedPlan), gate and up in float32 with f32_saved."""
    import torch

    xs, k, n = _product_sizes(xs, w_gate, rhs_transpose)
    plan = _product_plan(GatedPlan, k, n, activation, rhs_transpose, xs[0], f32_saved)
    tokens = len(xs) * xs[0].shape[0]
    gate = up = None
    with _On(stream):
        xs, (w_gate, w_up) = _shard_rows(xs), _pair_rows(w_gate, w_up)
        if out is None:
            out = torch.empty((tokens, n), dtype=xs[0].dtype, device=xs[0].device)
        if return_saved:
            gate, up = (torch.empty((tokens, n), dtype=plan._saved, device=xs[0].device) for _ in range(2))
        if workspace is None:
            workspace = plan.new_workspace()
    plan.run(xs, w_gate, w_up, out, workspace, gate=gate, up=up, stream=stream)
    return (out, gate, up) if return_saved else out


def gated_matmul_backward(d_out, xs, w_gate, w_up, gate, up, activation: str = "silu", rhs_transpose: bool = False,
                          f32_grads: bool = False, workspace=None, stream=None):
    """(dx, dw_gate, dw_up) of gated_matmul; gate and up as it saved them, in either type."""
    import torch

    xs, k, n = _product_sizes(xs, w_gate, rhs_transpose)
    plan = _product_plan(GatedPlan, k, n, activation, rhs_transpose, xs[0], gate.dtype is torch.float32)
    tokens = len(xs) * xs[0].shape[0]
    with _On(stream):
        xs, (w_gate, w_up), (gate, up) = _shard_rows(xs), _pair_rows(w_gate, w_up), _pair_rows(gate, up)
        d_out = _rows(d_out)
        d_gate, d_up = (torch.empty((tokens, n), dtype=xs[0].dtype, device=xs[0].device) for _ in range(2))
        dx = torch.empty((tokens, k), dtype=xs[0].dtype, device=xs[0].device)
        dw_gate, dw_up = (torch.empty(tuple(w_gate.shape), dtype=torch.float32 if f32_grads else xs[0].dtype, device=xs[0].device)
                          for _ in range(2))
        if workspace is None:
            workspace = plan.new_workspace()
    plan.backward(d_out, xs, w_gate, w_up, gate, up, d_gate, d_up, workspace, dx=dx, dw_gate=dw_gate, dw_up=dw_up, stream=stream)
    return dx, dw_gate, dw_up


def linear_matmul(xs, w, bias=None, residual=None, activation: Optional[str] = None, rhs_transpose: bool = False,
                  return_saved: bool = False, out=None, workspace=None, stream=None, f32_saved: bool = False):
    """act(X W + bias) + residual of X [tokens, k] or the shards of a gathered X;
    returns [tokens, n], with return_saved (out, pre) as the backward pass reads it
    (LinearPlan; without an activation pre is None: it reads nothing), pre in float32
    with f32_saved."""
    import torch

    xs, k, n = _product_sizes(xs, w, rhs_transpose)
    plan = _product_plan(LinearPlan, k, n, activation, rhs_transpose, xs[0], f32_saved)
    tokens = len(xs) * xs[0].shape[0]
    pre = None
    with _On(stream):
        xs, w, bias, residual = _shard_rows(xs), _rows(w), _vector(bias), _rows(residual)
        if out is None:
            out = torch.empty((tokens, n), dtype=xs[0].dtype, device=xs[0].device)
        if return_saved and activation is not None:
            pre = torch.empty((tokens, n), dtype=plan._saved, device=xs[0].device)
        if workspace is None:
            workspace = plan.new_workspace()
    plan.run(xs, w, out, workspace, bias=bias, residual=residual, pre=pre, stream=stream)
    return (out, pre) if return_saved else out


def linear_matmul_backward(d_out, xs, w, pre=None, activation: Optional[str] = None, rhs_transpose: bool = False,
                           f32_grads: bool = False, workspace=None, stream=None):
    """(dx, dw, d_bias) of linear_matmul, pre as it saved it, in either type; the
    residual's gradient is d_out."""
    import torch

    xs, k, n = _product_sizes(xs, w, rhs_transpose)
    plan = _product_plan(LinearPlan, k, n, activation, rhs_transpose, xs[0], pre is not None and pre.dtype is torch.float32)
    tokens = len(xs) * xs[0].shape[0]
    d_pre = None
    with _On(stream):
        xs, w, d_out, pre = _shard_rows(xs), _rows(w), _rows(d_out), _rows(pre)
        if activation is not None:
            d_pre = torch.empty((tokens, n), dtype=xs[0].dtype, device=xs[0].device)
        dx = torch.empty((tokens, k), dtype=xs[0].dtype, device=xs[0].device)
        grads = torch.float32 if f32_grads else xs[0].dtype
        dw = torch.empty(tuple(w.shape), dtype=grads, device=xs[0].device)
        d_bias = torch.empty(n, dtype=grads, device=xs[0].device)
        if workspace is None:
            workspace = plan.new_workspace()
    plan.backward(d_out, xs, w, workspace, pre=pre, d_pre=d_pre, dx=dx, dw=dw, d_bias=d_bias, stream=stream)
    return dx, dw, d_bias
