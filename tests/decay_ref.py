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


def _walk(x, y, z, g, S, back):
    """o_t = S_t^T x_t with S <- g_t S + y_t z_t^T; back: from the last token on, its decay applied once it has been
    read.  S is overwritten with the state at the end."""
    o = torch.empty(*x.shape[:3], z.shape[-1], dtype=torch.float64, device=x.device)
    for t in (range(x.shape[2] - 1, -1, -1) if back else range(x.shape[2])):
        if not back:
            S *= g[:, :, t, None, None]
        S += y[:, :, t, :, None] * z[:, :, t, None, :]
        o[:, :, t] = (x[:, :, t, None, :] @ S)[:, :, 0]
        if back:
            S *= g[:, :, t, None, None]
    return o


def walked_gradients(q, k, v, log_g, S0, dO, dS):
    """gradients() by the recurrence of dL/dS_t instead of autograd, for rows too long for it: with G_t = dL/dS_t =
    q_t dO_t^T + e^{l_{t+1}} G_{t+1}: dk_t = G_t v_t, dv_t = G_t^T k_t, dq_t = S_t dO_t, dl_t = e^{l_t} <G_t, S_{t-1}>
    = (q_t . dq_t + dl_{t+1}) - k_t . dk_t, and 0 where e^{l_t} is."""
    B, H, L, dk = q.shape
    q, k, v, dO = (t.double() for t in (q, k, v, dO))
    l = l64(log_g, B, L)
    g = torch.exp(l)
    shape = (B, H, dk, v.shape[-1])
    S = torch.zeros(shape, dtype=torch.float64, device=q.device) if S0 is None else S0.double()
    G = torch.zeros(shape, dtype=torch.float64, device=q.device) if dS is None else dS.double()
    St, Gt = S.transpose(2, 3).clone(), G.transpose(2, 3).clone()
    dq = _walk(dO, v, k, g, St, False)
    dk_ = _walk(v, dO, q, g, Gt, True)
    dS0 = G.clone()
    dv = _walk(k, q, dO, g, dS0, True)
    m = (q * dq).sum(-1) - (k * dk_).sum(-1)
    tail = (St.transpose(2, 3) * G).sum((2, 3))
    # sums from the end of each document: the running sum less what it was behind the next token that forgets
    s = m.flip(2).cumsum(2).flip(2) + tail[..., None]
    behind = torch.zeros_like(s)
    forgets = l < -200
    if bool(forgets.any()):
        at = torch.where(forgets, torch.arange(L, device=l.device), L).flip(2).cummin(2).values.flip(2)  # the next such token
        behind = torch.where(at < L, torch.gather(s, 2, at.clamp(max=L - 1)), 0.0)
    return dq, dk_, dv, torch.where(forgets, 0.0, s - behind), dS0
