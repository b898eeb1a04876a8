"""The gradients of decay_ref without autograd, for rows too long for it."""
import torch

from decay_ref import l64


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
    """decay_ref.gradients() by the recurrence of dL/dS_t instead of autograd, for rows too long for it: with G_t = dL/dS_t =
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
