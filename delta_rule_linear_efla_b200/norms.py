"""The norms around an attention of this library, which itself normalises nothing.

head_norm, before it: q or k out of a projection ([B,L,H,d], slices of a fused one included), each head
normalised, in the attention's layout [B,H,L,d].  gated_norm, after it: the readout [B,H,L,d], each head
normalised, gated, scaled and added to the residual, in the projections' layout [B,L,H,d].  Both are
differentiable; *_fwd and *_bwd are the plain calls.  efla_attention and decay_attention take them along.
Where a backward pass is captured into a CUDA graph, no eager autograd graph of the same leaves may be alive.
"""
from __future__ import annotations

import ctypes

import torch

from .decay import _arg, _launch_on, _workspace
from .efla import _check, _code, load_library

KINDS = {"l2": 0, "rms": 1}
ACTS = {"silu": 0, "sigmoid": 1}


def _option(table, name: str, value: str) -> int:
    if value not in table:
        raise ValueError("%s must be one of %s, got %r" % (name, sorted(table), value))
    return table[value]


def _view(t, name: str, device, shape, dtype):
    """(address, element strides) of a [B,L,H,d] tensor whose last dimension is dense."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.device != device:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, device))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    st = t.stride()
    if st[3] != 1 and shape[3] > 1:
        raise ValueError("%s must be dense in its last dimension" % name)
    return t.data_ptr(), (ctypes.c_longlong * 3)(*st[:3])


def _four(t, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dim() != 4:
        raise ValueError("%s must have 4 dimensions, got %d" % (name, t.dim()))
    return t.device, t.dtype, t.shape


def _weight(w, d, device):
    if w is None:
        return 0, 0
    return _arg(w, "weight", device, (d,), w.dtype if isinstance(w, torch.Tensor) else None), _code(w.dtype)


def head_norm_fwd(x, weight=None, kind: str = "l2", scale: float = 1.0, eps: float = 1e-6, y=None, stream=None):
    """y[b,h,t,:] = scale * weight * x[b,t,h,:] / sqrt(n + eps), n the sum ("l2") or the mean ("rms") of the
    row's squares.  x: [B,L,H,d] with a dense last dimension, float32 or bfloat16, d <= 256; weight: [d],
    float32 or bfloat16, or None; y: [B,H,L,d] in x's dtype."""
    device, dtype, (B, L, H, d) = _four(x, "x")
    xp, xs = _view(x, "x", device, x.shape, dtype)
    wp, wc = _weight(weight, d, device)
    with _launch_on(device, stream) as s:
        if y is None:
            y = torch.empty((B, H, L, d), dtype=dtype, device=device)
        _check(load_library().efla_head_norm(xp, xs, wp, wc, _arg(y, "y", device, (B, H, L, d), dtype), B, L, H, d,
                                             _code(dtype), _option(KINDS, "kind", kind), scale, eps, s), "efla_head_norm")
    return y


def head_norm_bwd(x, dy, weight=None, kind: str = "l2", scale: float = 1.0, eps: float = 1e-6, want_dw: bool = True,
                  workspace=None, stream=None):
    """(dx, dweight or None) of head_norm_fwd for dy [B,H,L,d]: dx dense in [B,L,H,d] and x's dtype, dweight in
    the weight's dtype."""
    device, dtype, (B, L, H, d) = _four(x, "x")
    xp, xs = _view(x, "x", device, x.shape, dtype)
    wp, wc = _weight(weight, d, device)
    dyp = _arg(dy, "dy", device, (B, H, L, d), dtype)
    if dy is None:
        raise ValueError("dy must be a CUDA tensor")
    lib = load_library()
    with _launch_on(device, stream) as s:
        dx = torch.empty((B, L, H, d), dtype=dtype, device=device)
        dw = torch.empty_like(weight) if weight is not None and want_dw else None
        ws, have = _workspace(workspace, lib.efla_norm_bwd_workspace_size(d) if dw is not None else 0, device)
        _check(lib.efla_head_norm_bwd(xp, xs, wp, wc, dyp, dx.data_ptr(), dw.data_ptr() if dw is not None else 0, B, L, H, d,
                                      _code(dtype), _option(KINDS, "kind", kind), scale, eps,
                                      ws.data_ptr() if ws is not None else 0, have, s), "efla_head_norm_bwd")
    return dx, dw


def gated_norm_fwd(o, gate, weight=None, residual=None, scale: float = 1.0, eps: float = 1e-6, act: str = "silu", y=None,
                   stream=None):
    """y[b,t,h,:] = residual[b,t,h,:] + scale * act(gate[b,t,h,:]) * weight * o[b,h,t,:] / sqrt(mean o^2 + eps).

    o: [B,H,L,d], float32 or bfloat16, d <= 256; gate: [B,L,H,d] with a dense last dimension, float32 or
    bfloat16; residual: like gate, or None; weight: [d], float32 or bfloat16, or None; act: "silu" or
    "sigmoid".  y: [B,L,H,d] in gate's dtype; it may be a dense residual."""
    device, o_dtype, (B, H, L, d) = _four(o, "o")
    dtype, shape = _four(gate, "gate")[1], (B, L, H, d)
    op = _arg(o, "o", device, (B, H, L, d), o_dtype)
    gp, gs = _view(gate, "gate", device, shape, dtype)
    rp, rs = _view(residual, "residual", device, shape, dtype) if residual is not None else (0, None)
    wp, wc = _weight(weight, d, device)
    with _launch_on(device, stream) as s:
        if y is None:
            y = torch.empty(shape, dtype=dtype, device=device)
        _check(load_library().efla_gated_norm(op, _code(o_dtype), gp, gs, wp, wc, rp, rs, _arg(y, "y", device, shape, dtype),
                                              B, L, H, d, _code(dtype), _option(ACTS, "act", act), scale, eps, s),
               "efla_gated_norm")
    return y


def gated_norm_bwd(o, gate, dy, weight=None, scale: float = 1.0, eps: float = 1e-6, act: str = "silu",
                   want_dw: bool = True, workspace=None, stream=None):
    """(do, dgate, dweight or None) of gated_norm_fwd for dy [B,L,H,d]; the residual's gradient is dy."""
    device, o_dtype, (B, H, L, d) = _four(o, "o")
    dtype, shape = _four(gate, "gate")[1], (B, L, H, d)
    op = _arg(o, "o", device, (B, H, L, d), o_dtype)
    gp, gs = _view(gate, "gate", device, shape, dtype)
    wp, wc = _weight(weight, d, device)
    if dy is None:
        raise ValueError("dy must be a CUDA tensor")
    dyp = _arg(dy, "dy", device, shape, dtype)
    lib = load_library()
    with _launch_on(device, stream) as s:
        do, dgate = torch.empty_like(o), torch.empty(shape, dtype=dtype, device=device)
        dw = torch.empty_like(weight) if weight is not None and want_dw else None
        ws, have = _workspace(workspace, lib.efla_norm_bwd_workspace_size(d) if dw is not None else 0, device)
        _check(lib.efla_gated_norm_bwd(op, _code(o_dtype), gp, gs, wp, wc, dyp, do.data_ptr(), dgate.data_ptr(),
                                       dw.data_ptr() if dw is not None else 0, B, L, H, d, _code(dtype),
                                       _option(ACTS, "act", act), scale, eps, ws.data_ptr() if ws is not None else 0, have,
                                       s), "efla_gated_norm_bwd")
    return do, dgate, dw


class HeadNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, kind, scale, eps):
        ctx.save_for_backward(x, weight)
        ctx.args = dict(kind=kind, scale=scale, eps=eps)
        return head_norm_fwd(x, weight, kind, scale, eps)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, weight = ctx.saved_tensors
        dx, dw = head_norm_bwd(x, dy.contiguous(), weight, want_dw=ctx.needs_input_grad[1], **ctx.args)
        return dx, dw, None, None, None


class GatedNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, o, gate, weight, residual, scale, eps, act):
        ctx.save_for_backward(o, gate, weight)
        ctx.args = dict(scale=scale, eps=eps, act=act)
        return gated_norm_fwd(o, gate, weight, residual, scale, eps, act)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        o, gate, weight = ctx.saved_tensors
        do, dgate, dw = gated_norm_bwd(o, gate, dy.contiguous(), weight, want_dw=ctx.needs_input_grad[2], **ctx.args)
        return do, dgate, dw, dy if ctx.needs_input_grad[3] else None, None, None, None


def head_norm(x, weight=None, kind: str = "l2", scale: float = 1.0, eps: float = 1e-6):
    """Differentiable head_norm_fwd."""
    return HeadNormFunction.apply(x, weight, kind, scale, eps)


def gated_norm(o, gate, weight=None, residual=None, scale: float = 1.0, eps: float = 1e-6, act: str = "silu"):
    """Differentiable gated_norm_fwd."""
    return GatedNormFunction.apply(o, gate, weight, residual, scale, eps, act)


def normed_attention(attention, q, k, qk_norm, gate, norm_weight, residual, scale, eps, act):
    """(o, S) of attention(q, k) with q and k normalised before it (qk_norm) and its output normalised, gated,
    scaled and added to the residual after it (gate)."""
    if gate is None and (norm_weight is not None or residual is not None or scale != 1.0):
        raise ValueError("norm_weight, residual and scale belong to the output's norm: give its gate")
    if qk_norm is not None:
        q, k = (head_norm(t.transpose(1, 2), kind=qk_norm, eps=eps) for t in (q, k))
    o, S = attention(q, k)
    if gate is not None:
        o = gated_norm(o, gate, norm_weight, residual, scale, eps, act)
    return o, S
