"""Operators around the losses: item embedding, log-probabilities over the whole
catalogue, and the policy and preference losses on them (include/rece.h).

Argument marshalling only, like the rest of the binding: every operator runs in
librece's HIP kernels, on torch's current stream of the tensors' device unless a
stream is given.  An operator object holds sizes and options, no device memory;
workspaces are allocated per call unless the caller passes one.  On a given stream
a call is that stream's work: what it allocates is that stream's memory, and memory
of its arguments and results that is freed waits for both streams.  Ordering the
streams (wait_stream, events) stays with the caller.
"""
from __future__ import annotations

import ctypes

from . import FLAG_BF16_GRADS, RECE_BF16, RECE_F32, _check, _ptr, lib

FLAG_ACCUMULATE, FLAG_NO_GRAD, FLAG_ENTROPY = 16, 32, 64
REDUCTIONS = {"token": 0, "sequence": 1}
PREFERENCE_KINDS = {"sigmoid": 0, "ipo": 1, "hinge": 2, "softmax": 3}


class PolicyConfig(ctypes.Structure):
    """Mirror of rece_policy_config in include/rece.h (field order and types)."""
    _fields_ = [("n", ctypes.c_int64), ("n_seq", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reduction", ctypes.c_int32), ("token_adv", ctypes.c_int32), ("clip_low", ctypes.c_float),
                ("clip_high", ctypes.c_float), ("kl_coef", ctypes.c_float), ("entropy_coef", ctypes.c_float)]


class PreferenceConfig(ctypes.Structure):
    """Mirror of rece_preference_config in include/rece.h (field order and types)."""
    _fields_ = [("n", ctypes.c_int64), ("n_seq", ctypes.c_int64), ("n_group", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("kind", ctypes.c_int32), ("average", ctypes.c_int32),
                ("beta", ctypes.c_float), ("margin", ctypes.c_float), ("smoothing", ctypes.c_float)]


def _dtype(name: str):
    if name not in ("bf16", "f32"):
        raise ValueError("dtype must be 'bf16' or 'f32'")
    import torch
    return (RECE_BF16, torch.bfloat16) if name == "bf16" else (RECE_F32, torch.float32)


def _want(name, t, dtype, shape, device=None):
    """Check one tensor argument: dtype, shape, contiguity, device."""
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor of shape {shape}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")


def _workspace(workspace, nbytes, device):
    """The caller's workspace, or a new one."""
    import torch
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if (workspace.device != device or workspace.numel() * workspace.element_size() < nbytes
            or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous buffer of at least {nbytes} bytes on {device}")
    return workspace


def _elsewhere(stream, device) -> bool:
    """Whether a stream is given that is not the device's current one."""
    import torch
    if stream is None:
        return False
    if stream.device != device:
        raise ValueError(f"stream must be a stream of {device}")
    return stream.cuda_stream != torch._C._cuda_getCurrentRawStream(device.index)


def _on_stream(stream, device, method, *args, **kw):
    """method(*args, **kw) with `stream` current: a workspace that is dropped on return is handed out again to that
    stream alone, and results lie in no memory that the caller's stream still uses."""
    import torch
    caller = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        out = method(*args, **kw)
    for t in (*args, *kw.values()):
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    for t in out if isinstance(out, tuple) else (out,):
        if t is not None:
            t.record_stream(caller)
    return out


def _call(fn, device, before, after):
    """fn(*before, stream, *after) with `device` current, on its current stream."""
    import torch
    index = device.index
    # the handle itself: torch.cuda.current_stream() makes an object around it, a third of a small call's time
    s = torch._C._cuda_getCurrentRawStream(index)
    if torch.cuda.current_device() == index:
        _check(fn(*before, s, *after))
        return
    with torch.cuda.device(device):
        _check(fn(*before, s, *after))


class ItemEmbedding:
    """Rows of an item table as a model's inputs (times `scale`) for n ids, and the
    table's gradient.  Ids outside [0, C) are padding: zero rows, no gradient.  For a bf16
    table trained through `embed` give bf16_grads=True: a float32 gradient (the default, for
    sums over several calls) is written whole and then converted by autograd."""

    def __init__(self, n: int, C: int, d: int, dtype: str = "bf16", scale: float = 1.0, bf16_grads: bool = False):
        self.n, self.C, self.d, self.dtype, self.scale = n, C, d, dtype, float(scale)
        self.bf16_grads = bool(bf16_grads)
        self._code, self._dt = _dtype(dtype)
        nb = ctypes.c_size_t()
        _check(lib().rece_embed_workspace_bytes(n, C, d, ctypes.byref(nb)))
        self.workspace_bytes = nb.value

    def forward(self, table, ids, out=None, stream=None):
        """Returns out [n, d] in the table's dtype."""
        import torch
        dev = table.device
        if _elsewhere(stream, dev):
            return _on_stream(stream, dev, self.forward, table, ids, out)
        _want("table", table, self._dt, (self.C, self.d))
        _want("ids", ids, torch.int32, (self.n,), dev)
        if out is None:
            out = torch.empty((self.n, self.d), dtype=self._dt, device=dev)
        else:
            _want("out", out, self._dt, (self.n, self.d), dev)
        _call(lib().rece_embed_forward, dev, (),
              (self.n, self.C, self.d, self._code, self.scale, _ptr(table), _ptr(ids), _ptr(out)))
        return out

    def backward(self, ids, dout, workspace=None, dtable=None, accumulate=False, stream=None):
        """Returns dtable [C, d] (float32, or bf16 with bf16_grads), every row written; with
        accumulate=True the gradient is added to the float32 dtable given."""
        import torch
        dev = dout.device
        if _elsewhere(stream, dev):
            return _on_stream(stream, dev, self.backward, ids, dout, workspace, dtable, accumulate)
        _want("dout", dout, self._dt, (self.n, self.d))
        _want("ids", ids, torch.int32, (self.n,), dev)
        gdt = torch.bfloat16 if self.bf16_grads else torch.float32
        if dtable is None:
            if accumulate:
                raise ValueError("accumulate needs the dtable to add to")
            dtable = torch.empty((self.C, self.d), dtype=gdt, device=dev)
        else:
            _want("dtable", dtable, gdt, (self.C, self.d), dev)
        ws = _workspace(workspace, self.workspace_bytes, dev)
        flags = (FLAG_BF16_GRADS if self.bf16_grads else 0) | (FLAG_ACCUMULATE if accumulate else 0)
        _call(lib().rece_embed_backward, dev, (),
              (self.n, self.C, self.d, self._code, self.scale, flags, _ptr(ids), _ptr(dout), _ptr(ws),
               ws.numel() * ws.element_size(), _ptr(dtable)))
        return dtable


class LogProb:
    """Log-probability of one item per position under the softmax over the whole
    catalogue (logits X Y^T / temperature), optionally the entropy of that softmax, and
    the gradients of both.  Ids outside [0, C) are padding: 0, no gradient.  For bf16 X and
    Y trained through `log_probs` give bf16_grads=True: float32 gradients (the default)
    take three products per weight instead of two, and autograd converts them."""

    def __init__(self, s: int, C: int, d: int, dtype: str = "bf16", temperature: float = 1.0, entropy: bool = False,
                 bf16_grads: bool = False):
        self.s, self.C, self.d, self.dtype = s, C, d, dtype
        self.temperature, self.entropy, self.bf16_grads = float(temperature), bool(entropy), bool(bf16_grads)
        self._code, self._dt = _dtype(dtype)
        self._flags = (FLAG_ENTROPY if entropy else 0) | (FLAG_BF16_GRADS if bf16_grads else 0)
        if not 2.0 ** -20 <= self.temperature <= 2.0 ** 64:
            raise ValueError("temperature must be positive, from 2^-20 to 2^64")
        self.workspace_bytes = self._bytes(self._flags)
        self.workspace_bytes_no_grad = self._bytes(self._flags | FLAG_NO_GRAD)

    def _bytes(self, flags):
        nb = ctypes.c_size_t()
        _check(lib().rece_logprob_workspace_bytes(self.s, self.C, self.d, self._code, flags, ctypes.byref(nb)))
        return nb.value

    def _check_inputs(self, X, Y, ids):
        import torch
        _want("X", X, self._dt, (self.s, self.d))
        _want("Y", Y, self._dt, (self.C, self.d), X.device)
        _want("ids", ids, torch.int32, (self.s,), X.device)

    def forward(self, X, Y, ids, workspace=None, need_grad=True, stream=None):
        """Returns (logp [s], entropy [s] or None, workspace); the workspace feeds backward
        (need_grad=False: it does not, and is smaller)."""
        import torch
        dev = X.device
        if _elsewhere(stream, dev):
            return _on_stream(stream, dev, self.forward, X, Y, ids, workspace, need_grad)
        self._check_inputs(X, Y, ids)
        flags = self._flags | (0 if need_grad else FLAG_NO_GRAD)
        ws = _workspace(workspace, self.workspace_bytes if need_grad else self.workspace_bytes_no_grad, dev)
        logp = torch.empty(self.s, dtype=torch.float32, device=dev)
        ent = torch.empty(self.s, dtype=torch.float32, device=dev) if self.entropy else None
        _call(lib().rece_logprob_forward, dev, (),
              (self.s, self.C, self.d, self._code, self.temperature, flags, _ptr(X), _ptr(Y), _ptr(ids), _ptr(ws),
               ws.numel() * ws.element_size(), _ptr(logp), _ptr(ent)))
        return logp, ent, ws

    def backward(self, X, Y, ids, workspace, dlogp, dentropy=None, dX=None, dY=None, stream=None):
        """Returns (dX [s, d], dY [C, d]): float32, or bf16 with bf16_grads.  `workspace` is the forward call's."""
        import torch
        if workspace is None:
            raise ValueError("workspace must be the one that forward returned (with need_grad)")
        dev = X.device
        if _elsewhere(stream, dev):
            return _on_stream(stream, dev, self.backward, X, Y, ids, workspace, dlogp, dentropy, dX, dY)
        self._check_inputs(X, Y, ids)
        gdt = torch.bfloat16 if self.bf16_grads else torch.float32
        _want("dlogp", dlogp, torch.float32, (self.s,), dev)
        if dentropy is not None:
            if not self.entropy:
                raise ValueError("dentropy needs entropy=True")
            _want("dentropy", dentropy, torch.float32, (self.s,), dev)
        if dX is None:
            dX = torch.empty((self.s, self.d), dtype=gdt, device=dev)
        if dY is None:
            dY = torch.empty((self.C, self.d), dtype=gdt, device=dev)
        _want("dX", dX, gdt, (self.s, self.d), dev)
        _want("dY", dY, gdt, (self.C, self.d), dev)
        ws = _workspace(workspace, self.workspace_bytes, dev)
        _call(lib().rece_logprob_backward, dev, (),
              (self.s, self.C, self.d, self._code, self.temperature, self._flags, _ptr(X), _ptr(Y), _ptr(ids), _ptr(ws),
               ws.numel() * ws.element_size(), _ptr(dlogp), _ptr(dentropy), _ptr(dX), _ptr(dY)))
        return dX, dY


class PolicyLoss:
    """Clipped policy loss with a KL and an entropy term over n_seq ragged sequences of
    n tokens in all, with the gradients in the same pass."""

    def __init__(self, n: int, n_seq: int, clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0,
                 entropy_coef: float = 0.0, reduction: str = "token", token_advantage: bool = False,
                 dtype: str = "f32"):
        if reduction not in REDUCTIONS:
            raise ValueError(f"reduction must be one of {sorted(REDUCTIONS)}")
        self._code, self._dt = _dtype(dtype)
        self.cfg = PolicyConfig(n, n_seq, self._code, REDUCTIONS[reduction], int(token_advantage), clip_low, clip_high,
                                kl_coef, entropy_coef)
        nb = ctypes.c_size_t()
        _check(lib().rece_policy_workspace_bytes(ctypes.byref(self.cfg), ctypes.byref(nb)))
        self.workspace_bytes = nb.value

    def forward(self, logp, old_logp, advantages, offsets, ref_logp=None, entropy=None, mask=None, dloss=None,
                workspace=None, grads=True, stream=None):
        """Returns (loss [1], stats [6], dlogp [n] or None, dentropy [n] or None); the
        gradients are those of dloss * loss (dloss a float32 tensor of one element, 1 if
        None), dentropy where an entropy is given.  grads=False computes none."""
        import torch
        c, dev = self.cfg, logp.device
        if _elsewhere(stream, dev):
            return _on_stream(stream, dev, self.forward, logp, old_logp, advantages, offsets, ref_logp, entropy, mask, dloss,
                              workspace, grads)
        n = (c.n,)
        for name, t in (("logp", logp), ("old_logp", old_logp), ("ref_logp", ref_logp), ("entropy", entropy)):
            if t is not None:
                _want(name, t, self._dt, n, dev)
        _want("advantages", advantages, torch.float32, (c.n if c.token_adv else c.n_seq,), dev)
        _want("offsets", offsets, torch.int32, (c.n_seq + 1,), dev)
        if mask is not None:
            if mask.dtype == torch.bool:
                mask = mask.view(torch.uint8)
            _want("mask", mask, torch.uint8, n, dev)
        if dloss is not None:
            _want("dloss", dloss, torch.float32, (1,), dev)
        ws = _workspace(workspace, self.workspace_bytes, dev)
        loss = torch.empty(1, dtype=torch.float32, device=dev)
        stats = torch.empty(6, dtype=torch.float32, device=dev)
        dlogp = torch.empty(n, dtype=self._dt, device=dev) if grads else None
        dent = torch.empty(n, dtype=self._dt, device=dev) if grads and entropy is not None else None
        _call(lib().rece_policy_loss, dev, (ctypes.byref(c),),
              (_ptr(logp), _ptr(old_logp), _ptr(ref_logp), _ptr(entropy), _ptr(advantages), _ptr(offsets), _ptr(mask),
               _ptr(dloss), _ptr(ws), ws.numel() * ws.element_size(), _ptr(loss), _ptr(stats), _ptr(dlogp),
               _ptr(dent)))
        return loss, stats, dlogp, dent


class PreferenceLoss:
    """Preference loss over n_group groups of sequences (the first of a group preferred),
    with the gradient in the same pass."""

    def __init__(self, n: int, n_seq: int, n_group: int, beta: float = 0.1, kind: str = "sigmoid",
                 label_smoothing: float = 0.0, margin: float = 0.0, average: bool = False, dtype: str = "f32"):
        if kind not in PREFERENCE_KINDS:
            raise ValueError(f"kind must be one of {sorted(PREFERENCE_KINDS)}")
        self._code, self._dt = _dtype(dtype)
        # label smoothing exists for the sigmoid kind alone
        smoothing = label_smoothing if kind == "sigmoid" else 0.0
        self.cfg = PreferenceConfig(n, n_seq, n_group, self._code, PREFERENCE_KINDS[kind], int(average), beta, margin,
                                    smoothing)
        nb = ctypes.c_size_t()
        _check(lib().rece_preference_workspace_bytes(ctypes.byref(self.cfg), ctypes.byref(nb)))
        self.workspace_bytes = nb.value

    def forward(self, logp, ref_logp, offsets, group_offsets, mask=None, dloss=None, workspace=None, grads=True,
                stream=None):
        """Returns (loss [1], loss_pg [n_group], rewards [n_seq], dlogp [n] or None); ref_logp
        None: a loss without a reference.  dlogp is the gradient of dloss * loss."""
        import torch
        c, dev = self.cfg, logp.device
        if _elsewhere(stream, dev):
            return _on_stream(stream, dev, self.forward, logp, ref_logp, offsets, group_offsets, mask, dloss, workspace, grads)
        n = (c.n,)
        _want("logp", logp, self._dt, n)
        if ref_logp is not None:
            _want("ref_logp", ref_logp, self._dt, n, dev)
        _want("offsets", offsets, torch.int32, (c.n_seq + 1,), dev)
        _want("group_offsets", group_offsets, torch.int32, (c.n_group + 1,), dev)
        if mask is not None:
            if mask.dtype == torch.bool:
                mask = mask.view(torch.uint8)
            _want("mask", mask, torch.uint8, n, dev)
        if dloss is not None:
            _want("dloss", dloss, torch.float32, (1,), dev)
        ws = _workspace(workspace, self.workspace_bytes, dev)
        loss = torch.empty(1, dtype=torch.float32, device=dev)
        out = torch.empty(c.n_group + c.n_seq, dtype=torch.float32, device=dev)
        loss_pg, rewards = out[:c.n_group], out[c.n_group:]
        dlogp = torch.empty(n, dtype=self._dt, device=dev) if grads else None
        _call(lib().rece_preference_loss, dev, (ctypes.byref(c),),
              (_ptr(logp), _ptr(ref_logp), _ptr(offsets), _ptr(group_offsets), _ptr(mask), _ptr(dloss), _ptr(ws),
               ws.numel() * ws.element_size(), _ptr(loss), _ptr(loss_pg), _ptr(rewards), _ptr(dlogp)))
        return loss, loss_pg, rewards, dlogp


# ------------------------------------------------------------------ autograd
_functions = {}


def _function(name):
    """The torch.autograd.Function of an operator (made at first use)."""
    if _functions:
        return _functions[name]
    import torch

    def scaled(grad, g):   # in bf16 a second rounding, unless g is a power of two
        return None if grad is None else (grad.float() * g).to(grad.dtype)

    class Embed(torch.autograd.Function):
        @staticmethod
        def forward(ctx, table, ids, op):
            ctx.op = op
            ctx.save_for_backward(ids)
            return op.forward(table, ids)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dout):
            (ids,) = ctx.saved_tensors
            dout = dout.contiguous()
            if dout.data_ptr() % 16:   # a part of a longer gradient (of a concatenation) may begin anywhere
                dout = dout.clone()
            return ctx.op.backward(ids, dout), None, None

    class LogProbs(torch.autograd.Function):
        @staticmethod
        def forward(ctx, X, Y, ids, op):
            logp, ent, ws = op.forward(X, Y, ids)
            ctx.op = op
            ctx.save_for_backward(X, Y, ids, ws)
            ctx.set_materialize_grads(False)
            return (logp, ent) if op.entropy else logp

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dlogp, dent=None):
            X, Y, ids, ws = ctx.saved_tensors
            if dlogp is None and dent is None:
                return None, None, None, None
            if dlogp is None:
                dlogp = torch.zeros_like(dent)
            dX, dY = ctx.op.backward(X, Y, ids, ws, dlogp.contiguous(), None if dent is None else dent.contiguous())
            return (dX if ctx.needs_input_grad[0] else None, dY if ctx.needs_input_grad[1] else None, None, None)

    class Policy(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logp, entropy, old, adv, offsets, ref, mask, op):
            loss, stats, dlogp, dent = op.forward(logp, old, adv, offsets, ref_logp=ref, entropy=entropy, mask=mask)
            ctx.save_for_backward(dlogp, dent)
            ctx.mark_non_differentiable(stats)
            return loss.squeeze_(), stats   # no view: a view made here could not be changed in place

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, g, _):
            dlogp, dent = ctx.saved_tensors
            return (scaled(dlogp, g), scaled(dent, g)) + (None,) * 6

    class Preference(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logp, ref, offsets, group_offsets, mask, op):
            loss, loss_pg, rewards, dlogp = op.forward(logp, ref, offsets, group_offsets, mask=mask)
            ctx.save_for_backward(dlogp)
            ctx.mark_non_differentiable(loss_pg, rewards)
            return loss.squeeze_(), loss_pg, rewards

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, g, *_):
            (dlogp,) = ctx.saved_tensors
            return (scaled(dlogp, g),) + (None,) * 5

    _functions.update(embed=Embed, log_probs=LogProbs, policy=Policy, preference=Preference)
    return _functions[name]


def _wanted(*tensors) -> bool:
    """Whether a gradient of some of these will be asked for (inside a Function the answer is lost: gradients are
    switched off there, and needs_input_grad stays set under no_grad)."""
    import torch
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def embed(table, ids, op: ItemEmbedding):
    """op.forward with autograd: the table's gradient is op.backward's."""
    return _function("embed").apply(table, ids, op)


def log_probs(X, Y, ids, op: LogProb):
    """logp [s] (and entropy [s] where op has it) with autograd for X and Y.  Where no gradient is wanted (no_grad, or
    neither requires one) the call computes and keeps nothing for it."""
    if not _wanted(X, Y):
        logp, ent, _ = op.forward(X, Y, ids, need_grad=False)
        return (logp, ent) if op.entropy else logp
    return _function("log_probs").apply(X, Y, ids, op)


def policy_loss(logp, old_logp, advantages, offsets, op: PolicyLoss, ref_logp=None, entropy=None, mask=None):
    """(mean loss, stats [6]) with autograd for logp and entropy."""
    if not _wanted(logp, entropy):
        loss, stats, _, _ = op.forward(logp, old_logp, advantages, offsets, ref_logp=ref_logp, entropy=entropy, mask=mask,
                                       grads=False)
        return loss.squeeze_(), stats
    return _function("policy").apply(logp, entropy, old_logp, advantages, offsets, ref_logp, mask, op)


def preference_loss(logp, ref_logp, offsets, group_offsets, op: PreferenceLoss, mask=None):
    """(mean loss, loss per group, rewards per sequence) with autograd for logp."""
    if not _wanted(logp):
        loss, loss_pg, rewards, _ = op.forward(logp, ref_logp, offsets, group_offsets, mask=mask, grads=False)
        return loss.squeeze_(), loss_pg, rewards
    return _function("preference").apply(logp, ref_logp, offsets, group_offsets, mask, op)
