"""Linear attention with a decay for each head: S_t = e^{l_t} S_{t-1} + k_t v_t^T, o_t = S_t^T q_t.

The prompt form (decay_chunk_fwd), its gradients (decay_bwd), one decode token (decay_recurrent_step) and
the differentiable call (decay_attention), bound to libefla.so like the delta rule's calls in `efla`: the
same layouts ([B,H,L,d]), the same float32 state, all computation in the library's kernels.

The log-decay l comes as [B,H,L] (one for every token, q's dtype) or as [H] float32 (one for each head).
It is expected to be <= 0; -inf forgets the state, so that the first token of each document packed into a
row carries -inf.
"""
from __future__ import annotations

import contextlib

import torch

from .efla import _check, _code, load_library

DECAY_TOKEN, DECAY_HEAD = 0, 1


@contextlib.contextmanager
def _switch(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream().cuda_stream
        else:  # outputs and workspaces are allocated for the stream that uses them
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


# The current stream's handle without the Stream object around it (3 us of a decode step's call), where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class _Here:
    """The current device's current stream: nothing to switch."""

    def __init__(self, index: int):
        self.index = index

    def __enter__(self):
        return _raw_stream(self.index) if _raw_stream else torch.cuda.current_stream().cuda_stream

    def __exit__(self, *exc):
        return False


_here: dict = {}


def _launch_on(device, stream):
    """Context in which a call on tensors of `device` allocates and launches; gives the stream's handle."""
    index = device.index
    if stream is None and index == torch.cuda.current_device():
        here = _here.get(index)
        if here is None:
            here = _here[index] = _Here(index)
        return here
    return _switch(device, stream)


def _arg(t, name: str, device, shape, dtype) -> int:
    """The address of a dense CUDA tensor of that device, shape and dtype (0 for None)."""
    if t is None:
        return 0
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.device != device:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, device))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _workspace(workspace, need: int, device):
    if not need:
        return None, 0
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on %s" % device)
    return workspace, workspace.numel() * workspace.element_size()


def _sizes(q, v, dim: int, name: str):
    for n, t in (("q", q), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError("%s must be a CUDA tensor" % n)
        if t.dim() != dim:
            raise ValueError("%s: %s must have %d dimensions, got %d" % (name, n, dim, t.dim()))
    return q.device, q.dtype, q.shape, v.shape[-1]


def _gate(log_g, shape, dtype, device):
    """(address, form) of the log-decays: `shape` in the input type or [H] float32."""
    if isinstance(log_g, torch.Tensor) and log_g.dim() == 1:
        return _arg(log_g, "log_g", device, (shape[1],), torch.float32), DECAY_HEAD
    if log_g is None:
        raise ValueError("log_g must be a CUDA tensor")
    return _arg(log_g, "log_g", device, shape, dtype), DECAY_TOKEN


def decay_workspace_size(B: int, H: int, L: int, dk: int, dv: int, dtype) -> int:
    return int(load_library().efla_decay_chunk_fwd_workspace_size(B, H, L, dk, dv, _code(dtype)))


def decay_chunk_fwd(q, k, v, log_g, S0=None, o=None, S_final=None, want_state: bool = True, workspace=None,
                    o_dtype=None, stream=None):
    """Forward over whole prompts.  Returns (o, S_final or None).

    q, k: [B,H,L,dk], v: [B,H,L,dv], all float32 or all bfloat16; log_g: [B,H,L] in their dtype or [H]
    float32; S0: [B,H,dk,dv] float32 or None for zeros.  o has q's dtype unless o_dtype (or o) says float32
    or bfloat16; S_final is float32 and may be S0 (in-place carry)."""
    device, dtype, shape, dv = _sizes(q, v, 4, "decay_chunk_fwd")
    B, H, L, dk = shape
    state, rows = (B, H, dk, dv), (B, H, L, dv)
    code = _code(dtype)
    o_dtype = o.dtype if o is not None else (o_dtype or dtype)
    qp, kp = _arg(q, "q", device, shape, dtype), _arg(k, "k", device, shape, dtype)
    vp, (gp, form) = _arg(v, "v", device, rows, dtype), _gate(log_g, (B, H, L), dtype, device)
    S0p = _arg(S0, "S0", device, state, torch.float32)
    lib = load_library()
    with _launch_on(device, stream) as s:
        if o is None:
            o = q.new_empty(rows, dtype=o_dtype)
        if S_final is None and want_state:
            S_final = q.new_empty(state, dtype=torch.float32)
        ws, have = _workspace(workspace, lib.efla_decay_chunk_fwd_workspace_size(B, H, L, dk, dv, code), device)
        _check(lib.efla_decay_chunk_fwd(qp, kp, vp, gp, form, S0p, _arg(o, "o", device, rows, o_dtype),
                                        _arg(S_final, "S_final", device, state, torch.float32), B, H, L, dk, dv, code,
                                        _code(o_dtype), ws.data_ptr() if ws is not None else 0, have, s),
               "efla_decay_chunk_fwd")
    return o, S_final


def decay_bwd(q, k, v, log_g, dO, S0=None, dS_final=None, want_dS0: bool = True, workspace=None, stream=None):
    """Gradients of decay_chunk_fwd: (dq, dk, dv, dlog_g, dS0) given dO = dL/do (q's dtype) and dS_final =
    dL/dS_final (float32 or None for 0).  dq, dk, dv and dlog_g have q's dtype, dS0 is float32.  dlog_g is
    None for a log_g of [H], which is a constant of the model; dS0 is None without want_dS0."""
    device, dtype, shape, dv = _sizes(q, v, 4, "decay_bwd")
    B, H, L, dk = shape
    state, rows = (B, H, dk, dv), (B, H, L, dv)
    code = _code(dtype)
    qp, kp = _arg(q, "q", device, shape, dtype), _arg(k, "k", device, shape, dtype)
    vp, (gp, form) = _arg(v, "v", device, rows, dtype), _gate(log_g, (B, H, L), dtype, device)
    dOp, S0p = _arg(dO, "dO", device, rows, dtype), _arg(S0, "S0", device, state, torch.float32)
    dSp = _arg(dS_final, "dS_final", device, state, torch.float32)
    lib = load_library()
    with _launch_on(device, stream) as s:
        dq, dkey, dval = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        dlog = torch.empty_like(log_g) if form == DECAY_TOKEN else None
        dS0 = q.new_empty(state, dtype=torch.float32) if want_dS0 else None
        ws, have = _workspace(workspace, lib.efla_decay_bwd_workspace_size(B, H, L, dk, dv, code), device)
        _check(lib.efla_decay_bwd(qp, kp, vp, gp, form, S0p, dOp, dSp, dq.data_ptr(), dkey.data_ptr(), dval.data_ptr(),
                                  dlog.data_ptr() if dlog is not None else 0, dS0.data_ptr() if want_dS0 else 0, B, H, L,
                                  dk, dv, code, ws.data_ptr() if ws is not None else 0, have, s), "efla_decay_bwd")
    return dq, dkey, dval, dlog, dS0


def decay_recurrent_step(q, k, v, log_g, S, o=None, o_dtype=None, stream=None):
    """One decode token per head: S ([B,H,dk,dv] float32) <- e^{log_g} S + k v^T in place; returns o = S^T q
    in q's dtype unless o_dtype (or o) says otherwise.  q, k: [B,H,dk], v: [B,H,dv]; log_g: [B,H] in their
    dtype or [H] float32; dk, dv <= 256."""
    device, dtype, shape, dv = _sizes(q, v, 3, "decay_recurrent_step")
    B, H, dk = shape
    o_dtype = o.dtype if o is not None else (o_dtype or dtype)
    if S is None:
        raise ValueError("S must be a CUDA tensor")
    code = _code(dtype)
    qp, kp = _arg(q, "q", device, shape, dtype), _arg(k, "k", device, shape, dtype)
    vp, (gp, form) = _arg(v, "v", device, (B, H, dv), dtype), _gate(log_g, (B, H), dtype, device)
    Sp = _arg(S, "S", device, (B, H, dk, dv), torch.float32)
    with _launch_on(device, stream) as s:
        if o is None:
            o = q.new_empty((B, H, dv), dtype=o_dtype)
        _check(load_library().efla_decay_recurrent_step(qp, kp, vp, gp, form, Sp, _arg(o, "o", device, (B, H, dv), o_dtype),
                                                        B, H, dk, dv, code, _code(o_dtype), s), "efla_decay_recurrent_step")
    return o


class DecayFunction(torch.autograd.Function):
    """(o, S_final) with gradients through efla_decay_bwd."""

    @staticmethod
    def forward(ctx, q, k, v, log_g, S0):
        o, S = decay_chunk_fwd(q, k, v, log_g, S0)
        ctx.save_for_backward(q, k, v, log_g, S0)
        ctx.set_materialize_grads(False)
        return o, S

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dO, dS):
        q, k, v, log_g, S0 = ctx.saved_tensors
        dO = torch.zeros_like(v) if dO is None else dO.contiguous()
        dS = None if dS is None else dS.contiguous()
        return decay_bwd(q, k, v, log_g, dO, S0, dS, want_dS0=ctx.needs_input_grad[4])


def decay_attention(q, k, v, log_g, S0=None, *, qk_norm: str | None = None, gate=None, norm_weight=None, residual=None,
                    scale: float = 1.0, eps: float = 1e-6, act: str = "silu"):
    """Differentiable decay_chunk_fwd: (o, S_final), with gradients to q, k, v, log_g ([B,H,L]) and S0.  A
    log_g of [H] is a constant of the model: one that requires a gradient is refused.  A learned one is given for every
    token, log_g[:, None].expand(B, H, L).to(q.dtype).contiguous(), and gets its gradient through that.

    qk_norm, gate, norm_weight, residual, scale, eps and act put the norms around it, as in
    efla.efla_attention; with a gate the output is [B,L,H,dv].

    A backward pass can be captured into a CUDA graph; no eager autograd graph of the same leaves may be alive
    then, since torch gathers a leaf's gradient on the stream of its first use, outside the capture."""
    from .norms import normed_attention

    if isinstance(log_g, torch.Tensor) and log_g.dim() == 1 and log_g.requires_grad:
        raise ValueError("log_g of [H] has no gradient: give one for every token, log_g[:, None].expand(B, H, L).to(q.dtype)"
                         ".contiguous()")
    return normed_attention(lambda q, k: DecayFunction.apply(q, k, v, log_g, S0), q, k, qk_norm, gate, norm_weight,
                            residual, scale, eps, act)
