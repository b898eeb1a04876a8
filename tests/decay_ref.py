"""Plain 64-bit forms of decayed linear attention and of the norms around it, for the tests: the token
recurrence and the formulas, differentiable by torch.autograd, with none of the library's code."""
import torch


def l64(log_g, B, L):
    """Log-decays as [B,H,L] float64."""
    l = log_g.double()
    return l[None, :, None].expand(B, l.shape[0], L) if l.dim() == 1 else l


def recurrence(q, k, v, log_g, S0=None):
    """S_t = e^{l_t} S_{t-1} + k_t v_t^T, o_t = S_t^T q_t: (o, S_L) in float64."""
    B, H, L, dk = q.shape
    q, k, v = q.double(), k.double(), v.double()
    g = torch.exp(l64(log_g, B, L))
    S = torch.zeros(B, H, dk, v.shape[-1], dtype=torch.float64, device=q.device) if S0 is None else S0.double()
    o = []
    for t in range(L):
        S = g[:, :, t, None, None] * S + k[:, :, t, :, None] * v[:, :, t, None, :]
        o.append((q[:, :, t, None, :] @ S)[:, :, 0])
    return (torch.stack(o, 2) if o else v[:, :, :0]), S


def gradients(q, k, v, log_g, S0, dO, dS):
    """Gradients of sum(o dO) + sum(S_L dS) by autograd through the recurrence: (dq, dk, dv, dlog_g, dS0)."""
    B, H, L, _ = q.shape
    leaves = [t.double().clone().requires_grad_(True) for t in (q, k, v)]
    l = l64(log_g, B, L).clone().requires_grad_(True)
    S = torch.zeros(B, H, q.shape[-1], v.shape[-1], dtype=torch.float64, device=q.device) if S0 is None else S0.double()
    S = S.clone().requires_grad_(True)
    o, Sf = recurrence(*leaves, l, S)
    loss = (o * dO.double()).sum() + (0.0 if dS is None else (Sf * dS.double()).sum())
    return torch.autograd.grad(loss, leaves + [l, S])


def head_norm(x, w, kind, scale, eps):
    x = x.double()
    n = x.square().sum(-1, keepdim=True) if kind == "l2" else x.square().mean(-1, keepdim=True)
    y = scale * x / torch.sqrt(n + eps)
    return (y if w is None else y * w.double()).transpose(1, 2)


def gated_norm(o, gate, w, residual, scale, eps, act):
    o, gate = o.double().transpose(1, 2), gate.double()
    a = torch.sigmoid(gate) * (gate if act == "silu" else 1.0)
    y = scale * a * o / torch.sqrt(o.square().mean(-1, keepdim=True) + eps)
    y = y if w is None else y * w.double()
    return y if residual is None else y + residual.double()


def far(x, ref):
    """(relative error in the 2-norm, largest error over max(rms, |ref|)) of a result; both 0 for no elements."""
    x, ref = x.detach().double(), ref.detach().double().to(x.device)
    assert x.shape == ref.shape and torch.isfinite(x).all() and torch.isfinite(ref).all()
    if not x.numel():
        return 0.0, 0.0
    d, norm = x - ref, ref.norm()
    if norm == 0:
        return float(d.norm()), float(d.abs().max())
    rms = norm / ref.numel() ** 0.5
    return float(d.norm() / norm), float((d.abs() / torch.maximum(ref.abs(), rms)).max())
