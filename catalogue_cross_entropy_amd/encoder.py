"""Operators of the sequence encoder between the item embedding and the loss, and of
scoring the catalogue in 8 bits (include/rece.h): causal attention over packed
sequences with a learned bias by buckets of the distance, the same for the last token
of every sequence over a cache, the residual root-mean-square norm, rows in 8 bits and
their scores.

Argument marshalling only, like the rest of the binding; what ops.py says about streams
and workspaces holds here too.

Every call can be captured into a graph.  For autograd's backward pass torch asks that no
eager graph over the same leaves is alive during the capture (their gradients' nodes belong
to the eager stream, and torch ends the process): drop its results first, or warm up on the
stream of the capture.
"""
from __future__ import annotations

import ctypes

from . import _check, _ptr, lib
from .ops import _call, _dtype, _elsewhere, _on_stream, _wanted, _want, _workspace

MAX_BOUNDS, MAX_DISTANCE = 127, 4096


class AttentionConfig(ctypes.Structure):
    """Mirror of rece_attention_config in include/rece.h (field order and types)."""
    _fields_ = [("n", ctypes.c_int64), ("n_seq", ctypes.c_int64), ("q_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("n_bounds", ctypes.c_int32), ("bounds", ctypes.c_int32 * MAX_BOUNDS)]


def log_buckets(n_buckets: int, max_distance: int = 128):
    """Bounds of n_buckets buckets of distances: the lower half one distance each (0, 1, 2, ...), the upper half
    by equal ratios up to max_distance, from where on there is one bucket.  `bounds` of the attention operators."""
    half = n_buckets // 2
    if n_buckets < 2 or n_buckets % 2 or not half < max_distance <= MAX_DISTANCE or n_buckets - 1 > MAX_BOUNDS:
        raise ValueError(f"n_buckets must be even, from 2 to {MAX_BOUNDS + 1}, max_distance from n_buckets / 2 + 1 to "
                         f"{MAX_DISTANCE}")
    bounds = list(range(1, half + 1))
    for k in range(1, half):
        # the first t with (t / half) ** half >= (max_distance / half) ** k, in whole numbers
        t, goal = bounds[-1] + 1, half ** (half - k) * max_distance ** k
        while t ** half < goal:
            t += 1
        bounds.append(t)
    return bounds


class _Attention:
    """What the two attention operators share: sizes, head layout, buckets."""

    def __init__(self, rows, n_seq, heads, d, kv_heads, dtype, scale, bounds):
        kv_heads = heads if kv_heads is None else kv_heads
        self.n_seq, self.heads, self.kv_heads, self.d, self.dtype = n_seq, heads, kv_heads, d, dtype
        self.scale = d ** -0.5 if scale is None else float(scale)
        self.bounds = None if bounds is None else [int(b) for b in bounds]
        self._code, self._dt = _dtype(dtype)
        if bounds is not None and len(self.bounds) > MAX_BOUNDS:
            raise ValueError(f"at most {MAX_BOUNDS} bounds")
        if bounds is not None and any(not 1 <= b <= MAX_DISTANCE for b in self.bounds):
            raise ValueError(f"bounds must be in [1, {MAX_DISTANCE}]")
        self._rows = rows
        self._cfgs = {}
        self.cfg = self._config(heads * d, kv_heads * d, kv_heads * d)

    def _config(self, *strides):
        """The configuration with these row strides (few ever occur)."""
        c = self._cfgs.get(strides)
        if c is None:
            b = self.bounds or []
            c = AttentionConfig(self._rows, self.n_seq, *strides, self.heads, self.kv_heads, self.d, self._code, self.scale,
                                len(b), (ctypes.c_int32 * MAX_BOUNDS)(*b))
            if len(self._cfgs) < 64:
                self._cfgs[strides] = c
        return c

    def _heads(self, name, t, rows, heads, device=None):
        """Check rows of heads (a slice of a wider projection will do); returns the stride of its rows."""
        d, at = self.d, t.stride()
        if (t.dtype is not self._dt or t.shape != (rows, heads, d) or not t.is_cuda or at[2] != 1
                or (heads > 1 and at[1] != d)):
            raise ValueError(f"{name} must be a CUDA {self._dt} tensor of shape {(rows, heads, d)} whose rows are "
                             "contiguous")
        if device is not None and t.device != device:
            raise ValueError(f"{name} must be on {device}")
        return at[0] if rows > 1 else heads * d

    def _bias(self, bias, device):
        import torch
        if (bias is None) != (self.bounds is None):
            raise ValueError("bias goes with an operator that has bounds")
        if bias is not None:
            _want("bias", bias, torch.float32, (len(self.bounds) + 1, self.heads), device)


class SequenceAttention(_Attention):
    """Causal attention over n_seq packed sequences of n tokens in all, `heads` query heads and `kv_heads` key
    heads of d elements, scores scaled by `scale` (default d ** -0.5).  With `bounds` (see log_buckets) a learned
    bias[len(bounds) + 1, heads] is added to the scores by the distance between query and key."""

    def __init__(self, n: int, n_seq: int, heads: int, d: int, kv_heads: int = None, dtype: str = "bf16",
                 scale: float = None, bounds=None):
        super().__init__(n, n_seq, heads, d, kv_heads, dtype, scale, bounds)
        self.n = n
        nb = ctypes.c_size_t()
        _check(lib().rece_attention_workspace_bytes(ctypes.byref(self.cfg), ctypes.byref(nb)))
        self.workspace_bytes = nb.value

    def _check_inputs(self, q, k, v, offsets, bias):
        import torch
        strides = (self._heads("q", q, self.n, self.heads), self._heads("k", k, self.n, self.kv_heads, q.device),
                   self._heads("v", v, self.n, self.kv_heads, q.device))
        _want("offsets", offsets, torch.int32, (self.n_seq + 1,), q.device)
        self._bias(bias, q.device)
        return self._config(*strides)

    def forward(self, q, k, v, offsets, bias=None, out=None, workspace=None, need_grad=True, stream=None):
        """Returns (out [n, heads, d], workspace); the workspace feeds backward (need_grad=False: None)."""
        import torch
        dev = q.device
        if _elsewhere(stream, dev):
            return _on_stream(stream, dev, self.forward, q, k, v, offsets, bias, out, workspace, need_grad)
        c = self._check_inputs(q, k, v, offsets, bias)
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        else:
            _want("out", out, self._dt, (self.n, self.heads, self.d), dev)
        ws = _workspace(workspace, self.workspace_bytes, dev) if need_grad else None
        _call(lib().rece_attention_forward, dev, (ctypes.byref(c),),
              (_ptr(q), _ptr(k), _ptr(v), _ptr(offsets), _ptr(bias), _ptr(ws),
               0 if ws is None else ws.numel() * ws.element_size(), _ptr(out)))
        return out, ws

    def backward(self, q, k, v, offsets, out, workspace, dout, bias=None, dq=None, dk=None, dv=None, stream=None):
        """Returns (dq, dk, dv, dbias or None); dq, dk and dv may be given as slices of one gradient.  `out` and
        `workspace` are those of the forward call."""
        import torch
        if workspace is None:
            raise ValueError("workspace must be the one that forward returned (with need_grad)")
        dev = q.device
        if _elsewhere(stream, dev):
            return _on_stream(stream, dev, self.backward, q, k, v, offsets, out, workspace, dout, bias, dq, dk, dv)
        c = self._check_inputs(q, k, v, offsets, bias)
        shape = (self.n, self.heads, self.d)
        _want("out", out, self._dt, shape, dev)
        _want("dout", dout, self._dt, shape, dev)
        grads = []
        for name, t, like, heads in (("dq", dq, q, self.heads), ("dk", dk, k, self.kv_heads), ("dv", dv, v, self.kv_heads)):
            if t is None:
                grads.append((torch.empty_like(like, memory_format=torch.contiguous_format), heads * self.d))
            else:
                grads.append((t, self._heads(name, t, self.n, heads, dev)))
        dbias = None if bias is None else torch.empty_like(bias)
        ws = _workspace(workspace, self.workspace_bytes, dev)
        (dq, sq), (dk, sk), (dv, sv) = grads
        _call(lib().rece_attention_backward, dev, (ctypes.byref(c),),
              (_ptr(q), _ptr(k), _ptr(v), _ptr(offsets), _ptr(bias), _ptr(out), _ptr(ws), ws.numel() * ws.element_size(),
               _ptr(dout), sq, sk, sv, _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dbias)))
        return dq, dk, dv, dbias


class LastAttention(_Attention):
    """Attention of the last token of each of n_seq sequences over a cache of `rows` rows of keys and values:
    sequence u's are rows begin[u] .. begin[u] + length[u] - 1 (packed histories, or slots of a cache that
    grows).  `max_len`: the lengths to plan for.  Otherwise as SequenceAttention, forward only."""

    def __init__(self, n_seq: int, rows: int, heads: int, d: int, max_len: int, kv_heads: int = None, dtype: str = "bf16",
                 scale: float = None, bounds=None):
        super().__init__(rows, n_seq, heads, d, kv_heads, dtype, scale, bounds)
        self.rows, self.max_len = rows, max_len
        nb = ctypes.c_size_t()
        _check(lib().rece_last_attention_workspace_bytes(ctypes.byref(self.cfg), max_len, ctypes.byref(nb)))
        self.workspace_bytes = nb.value

    def forward(self, q, k, v, begin, length, bias=None, out=None, workspace=None, stream=None):
        """Returns out [n_seq, heads, d]; q [n_seq, heads, d], k and v [rows, kv_heads, d]."""
        import torch
        dev = q.device
        if _elsewhere(stream, dev):
            return _on_stream(stream, dev, self.forward, q, k, v, begin, length, bias, out, workspace)
        c = self._config(self._heads("q", q, self.n_seq, self.heads), self._heads("k", k, self.rows, self.kv_heads, dev),
                         self._heads("v", v, self.rows, self.kv_heads, dev))
        _want("begin", begin, torch.int32, (self.n_seq,), dev)
        _want("length", length, torch.int32, (self.n_seq,), dev)
        self._bias(bias, dev)
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        else:
            _want("out", out, self._dt, (self.n_seq, self.heads, self.d), dev)
        ws = _workspace(workspace, self.workspace_bytes, dev) if self.workspace_bytes else None
        _call(lib().rece_last_attention, dev, (ctypes.byref(c),),
              (self.max_len, _ptr(q), _ptr(k), _ptr(v), _ptr(begin), _ptr(length), _ptr(bias), _ptr(ws),
               0 if ws is None else ws.numel() * ws.element_size(), _ptr(out)))
        return out


class ResidualNorm:
    """Root-mean-square norm of n rows of d elements after the addition of a branch to the residual stream:
    h = x + residual, y = h / sqrt(mean h^2 + eps) * weight (weight float32), or y in 8 bits with a scale per row."""

    def __init__(self, n: int, d: int, eps: float = 1e-6, dtype: str = "bf16"):
        self.n, self.d, self.eps, self.dtype = n, d, float(eps), dtype
        self._code, self._dt = _dtype(dtype)
        if not 0.0 <= self.eps < float("inf"):
            raise ValueError("eps must be finite and >= 0")
        nb = ctypes.c_size_t()
        _check(lib().rece_norm_workspace_bytes(n, d, ctypes.byref(nb)))
        self.workspace_bytes = nb.value

    def _check_inputs(self, x, residual, weight, h):
        """Returns the h to write (None without a residual, unless one is given)."""
        import torch
        _want("x", x, self._dt, (self.n, self.d))
        _want("weight", weight, torch.float32, (self.d,), x.device)
        if residual is not None:
            _want("residual", residual, self._dt, (self.n, self.d), x.device)
            if h is None:
                return torch.empty_like(x)
        if h is not None:
            _want("h", h, self._dt, (self.n, self.d), x.device)
        return h

    def forward(self, x, residual, weight, h=None, stream=None):
        """Returns (y, h, rstd); h is x itself without a residual.  `h` may be given, x or residual itself too."""
        import torch
        dev = x.device
        if _elsewhere(stream, dev):
            return _on_stream(stream, dev, self.forward, x, residual, weight, h)
        h = self._check_inputs(x, residual, weight, h)
        y = torch.empty_like(x)
        rstd = torch.empty(self.n, dtype=torch.float32, device=dev)
        _call(lib().rece_norm_forward, dev, (),
              (self.n, self.d, self._code, self.eps, _ptr(x), _ptr(residual), _ptr(weight), _ptr(h), _ptr(y), _ptr(rstd)))
        return y, x if h is None else h, rstd

    def forward_int8(self, x, residual, weight, h=None, stream=None):
        """Returns (y8 [n, d] int8, scale [n], h): y = y8 * scale of the row."""
        import torch
        dev = x.device
        if _elsewhere(stream, dev):
            return _on_stream(stream, dev, self.forward_int8, x, residual, weight, h)
        h = self._check_inputs(x, residual, weight, h)
        y8 = torch.empty_like(x, dtype=torch.int8)
        scale = torch.empty(self.n, dtype=torch.float32, device=dev)
        _call(lib().rece_norm_forward_int8, dev, (),
              (self.n, self.d, self._code, self.eps, _ptr(x), _ptr(residual), _ptr(weight), _ptr(h), _ptr(y8), _ptr(scale)))
        return y8, scale, x if h is None else h

    def backward(self, dy, h, weight, rstd, dh=None, workspace=None, stream=None):
        """Returns (dx, dweight): dx is the gradient of x and of the residual; dh that of h from past the norm."""
        import torch
        dev = dy.device
        if _elsewhere(stream, dev):
            return _on_stream(stream, dev, self.backward, dy, h, weight, rstd, dh, workspace)
        shape = (self.n, self.d)
        _want("dy", dy, self._dt, shape)
        _want("h", h, self._dt, shape, dev)
        if dh is not None:
            _want("dh", dh, self._dt, shape, dev)
        _want("weight", weight, torch.float32, (self.d,), dev)
        _want("rstd", rstd, torch.float32, (self.n,), dev)
        ws = _workspace(workspace, self.workspace_bytes, dev)
        dx, dw = torch.empty_like(dy), torch.empty_like(weight)
        _call(lib().rece_norm_backward, dev, (),
              (self.n, self.d, self._code, _ptr(dy), _ptr(h), _ptr(dh), _ptr(weight), _ptr(rstd), _ptr(ws),
               ws.numel() * ws.element_size(), _ptr(dx), _ptr(dw)))
        return dx, dw


def quantize_rows(x, stream=None):
    """Rows of a float32 or bf16 [n, d] tensor in 8 bits: (x8 int8, scale [n] float32), x = x8 * scale of the row."""
    import torch
    dev = x.device
    if _elsewhere(stream, dev):
        return _on_stream(stream, dev, quantize_rows, x)
    code, dt = _dtype("f32" if x.dtype == torch.float32 else "bf16")
    if x.dim() != 2:
        raise ValueError("x must have two dimensions")
    _want("x", x, dt, x.shape)
    x8 = torch.empty_like(x, dtype=torch.int8)
    scale = torch.empty(x.shape[0], dtype=torch.float32, device=dev)
    _call(lib().rece_quantize_rows, dev, (), (x.shape[0], x.shape[1], code, _ptr(x), _ptr(x8), _ptr(scale)))
    return x8, scale


class Int8Scores:
    """Scores of s positions against C items, both as rows of d 8-bit integers with a float32 scale each
    (quantize_rows, ResidualNorm.forward_int8), d a multiple of 16, in bf16 or float32."""

    def __init__(self, s: int, C: int, d: int, dtype: str = "bf16"):
        self.s, self.C, self.d, self.dtype = s, C, d, dtype
        self._code, self._dt = _dtype(dtype)
        if s < 0 or C < 1 or d < 16 or d % 16 or d > 8192:
            raise ValueError("s must be >= 0, C >= 1, d a multiple of 16, at most 8192")

    def forward(self, x8, sx, y8, sy, out=None, stream=None):
        """Returns out [s, C] = (x8 y8^T) sx sy."""
        import torch
        dev = x8.device
        if _elsewhere(stream, dev):
            return _on_stream(stream, dev, self.forward, x8, sx, y8, sy, out)
        _want("x8", x8, torch.int8, (self.s, self.d))
        _want("y8", y8, torch.int8, (self.C, self.d), dev)
        _want("sx", sx, torch.float32, (self.s,), dev)
        _want("sy", sy, torch.float32, (self.C,), dev)
        if out is None:
            out = torch.empty((self.s, self.C), dtype=self._dt, device=dev)
        else:
            _want("out", out, self._dt, (self.s, self.C), dev)
        _call(lib().rece_int8_scores, dev, (),
              (self.s, self.C, self.d, self._code, _ptr(x8), _ptr(sx), _ptr(y8), _ptr(sy), _ptr(out)))
        return out


# ------------------------------------------------------------------ autograd
_functions = {}


def _function(name):
    """The torch.autograd.Function of an operator (made at first use)."""
    if _functions:
        return _functions[name]
    import torch

    def laid_out(g):   # a part of a longer gradient (of a concatenation) may begin anywhere
        g = g.contiguous()
        return g.clone() if g.data_ptr() % 16 else g

    class Attention(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, bias, offsets, op):
            out, ws = op.forward(q, k, v, offsets, bias=bias)
            ctx.op = op
            ctx.save_for_backward(q, k, v, bias, offsets, out, ws)
            return out

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dout):
            q, k, v, bias, offsets, out, ws = ctx.saved_tensors
            grads = ctx.op.backward(q, k, v, offsets, out, ws, laid_out(dout), bias=bias)
            return tuple(g if need else None for g, need in zip(grads, ctx.needs_input_grad)) + (None, None)

    class AttentionQkv(torch.autograd.Function):
        @staticmethod
        def forward(ctx, qkv, bias, offsets, op):
            out, ws = op.forward(*_split(qkv, op), offsets, bias=bias)
            ctx.op = op
            ctx.save_for_backward(qkv, bias, offsets, out, ws)
            return out

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dout):
            qkv, bias, offsets, out, ws = ctx.saved_tensors
            dqkv = torch.empty(qkv.shape, dtype=qkv.dtype, device=qkv.device)
            dq, dk, dv = _split(dqkv, ctx.op)
            *_, dbias = ctx.op.backward(*_split(qkv, ctx.op), offsets, out, ws, laid_out(dout), bias=bias, dq=dq, dk=dk,
                                        dv=dv)
            return dqkv, dbias if ctx.needs_input_grad[1] else None, None, None

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, residual, weight, op):
            y, h, rstd = op.forward(x, residual, weight)
            ctx.op = op
            ctx.save_for_backward(h, weight, rstd)
            ctx.set_materialize_grads(False)
            return y if residual is None else (y, h)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dy, dh=None):
            h, weight, rstd = ctx.saved_tensors
            if dy is None:
                dx, dw = dh, None
            else:
                dx, dw = ctx.op.backward(laid_out(dy), h, weight, rstd, dh=None if dh is None else laid_out(dh))
            need = ctx.needs_input_grad
            return dx if need[0] else None, dx if need[1] else None, dw if need[2] else None, None

    _functions.update(attention=Attention, attention_qkv=AttentionQkv, norm=Norm)
    return _functions[name]


def _split(qkv, op):
    """q, k and v as slices of one projection [n, (heads + 2 kv_heads) * d]."""
    a, b, d = op.heads * op.d, (op.heads + op.kv_heads) * op.d, op.d
    n = qkv.shape[0]
    return (qkv[:, :a].view(n, op.heads, d), qkv[:, a:b].view(n, op.kv_heads, d), qkv[:, b:].view(n, op.kv_heads, d))


def attention(q, k, v, offsets, op: SequenceAttention, bias=None):
    """out [n, heads, d] with autograd for q, k, v and the bias."""
    if not _wanted(q, k, v, bias):
        return op.forward(q, k, v, offsets, bias=bias, need_grad=False)[0]
    return _function("attention").apply(q, k, v, bias, offsets, op)


def attention_qkv(qkv, offsets, op: SequenceAttention, bias=None):
    """The same from one projection [n, (heads + 2 kv_heads) * d] (queries, keys, values), whose gradient is written
    in one piece."""
    if qkv.dim() != 2 or qkv.shape[1] != (op.heads + 2 * op.kv_heads) * op.d or qkv.stride(1) != 1:
        raise ValueError(f"qkv must be rows of {(op.heads + 2 * op.kv_heads) * op.d} contiguous elements")
    if not _wanted(qkv, bias):
        return op.forward(*_split(qkv, op), offsets, bias=bias, need_grad=False)[0]
    return _function("attention_qkv").apply(qkv, bias, offsets, op)


def residual_norm(x, residual, weight, op: ResidualNorm):
    """(y, h) with autograd for x, the residual and the weight; residual None: (y, x)."""
    if not _wanted(x, residual, weight):
        return op.forward(x, residual, weight)[:2]
    out = _function("norm").apply(x, residual, weight, op)
    return (out, x) if residual is None else out
