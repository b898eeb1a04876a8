"""The operators of a decayed linear-attention layer, as they are measured: plain forms in elementary torch
operations and the library's own calls on the same inputs.

  fwd    decayed linear attention over a prompt: S_t = e^{l_t} S_{t-1} + k_t v_t^T, o_t = S_t^T q_t
  bwd    its gradients
  step   one decode token, the state updated in place
  hnorm  the per-head norm of q or k before the attention (projection layout to head layout)
  gnorm  the per-head norm of the readout after it, with output gate, residual scale and residual

Layouts: q, k [B,H,L,dk], v, o [B,H,L,dv], l [B,H,L] in the input type or [H] float32 (a fixed decay for each head);
states [B,H,dk,dv] float32; projections and gates [B,L,H,d], slices of one fused projection where a layer has one.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # prefill of the 1.3B-shaped workload, a learned decay for every token
        dict(name="prefill_1p3b", op="fwd", dtype="bf16", B=4, H=16, L=4096, dk=128, dv=128, decay="token", s0=False, docs=0),
        # one long prompt, a fixed decay for each head
        dict(name="prefill_long", op="fwd", dtype="bf16", B=1, H=16, L=65536, dk=128, dv=128, decay="head", s0=False, docs=0),
        # a short float32 prompt of odd sizes continued from a state, with several documents in it
        dict(name="prefill_odd_fp32", op="fwd", dtype="fp32", B=2, H=3, L=777, dk=48, dv=80, decay="token", s0=True, docs=5),
        # training: gradients of the 340M-shaped workload
        dict(name="train_340m", op="bwd", dtype="bf16", B=8, H=8, L=2048, dk=128, dv=128, decay="token", s0=False, docs=0),
        # training: gradients of the 1.3B-shaped workload, documents packed into its rows
        dict(name="train_1p3b", op="bwd", dtype="bf16", B=4, H=16, L=4096, dk=128, dv=128, decay="token", s0=False, docs=3),
        # training in float32, ragged, through an initial state
        dict(name="train_ragged_fp32", op="bwd", dtype="fp32", B=1, H=4, L=500, dk=64, dv=64, decay="token", s0=True, docs=0),
        # the decode batch of the 1.3B-shaped workload
        dict(name="decode_1p3b", op="step", dtype="bf16", B=64, H=16, dk=128, dv=128, decay="token"),
        # one sequence's decode step: latency
        dict(name="decode_one", op="step", dtype="fp32", B=1, H=8, dk=64, dv=64, decay="head"),
        # q or k of a training step out of a fused projection, with the norm's gradients
        dict(name="norm_in_train", op="hnorm", dtype="bf16", B=4, L=4096, H=16, d=128, kind="l2", weight=True, fused=3, train=True),
        # a short float32 batch at an odd head size
        dict(name="norm_in_odd_fp32", op="hnorm", dtype="fp32", B=2, L=333, H=5, d=80, kind="rms", weight=True, fused=1, train=True),
        # the readout of a training step, gated, scaled and added to the residual, with its gradients
        dict(name="norm_out_train", op="gnorm", dtype="bf16", B=4, L=4096, H=16, d=128, act="silu", weight=True, residual=True, fused=2, train=True),
        # the readout of one decode step
        dict(name="norm_out_decode", op="gnorm", dtype="bf16", B=64, L=1, H=16, d=128, act="silu", weight=True, residual=False, fused=1, train=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("fwd", "fwd", "bwd", "bwd", "step", "hnorm", "gnorm"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    if op in ("fwd", "bwd"):
        if dtype == "bf16" and rng.random() < 0.7:
            dk, dv = rng.choice((64, 128)), rng.choice((64, 128))
        else:
            dk, dv = rng.randint(8, 128), rng.randint(8, 128)
        fast = dtype == "bf16" and dk % 64 == 0 and dv % 64 == 0
        most = (1 << 20 if op == "fwd" else 1 << 18) if fast else 1 << 16
        H = rng.choice((1, 2, 3, 4, 8, 16, 20, 32))
        B = rng.choice((1, 1, 2, 3, 4, 8))
        L = _log_int(rng, 1, max(1, most // (B * H)))
        decay = "head" if rng.random() < 0.3 else "token"
        return dict(op=op, dtype=dtype, B=B, H=H, L=L, dk=dk, dv=dv, decay=decay, s0=rng.random() < 0.5,
                    docs=rng.randint(1, 6) if decay == "token" and rng.random() < 0.4 else 0)
    if op == "step":
        d = (rng.choice((64, 128)), rng.choice((64, 128))) if rng.random() < 0.7 else (rng.randint(4, 256), rng.randint(4, 256))
        H = rng.choice((1, 2, 4, 8, 12, 16, 32))
        B = _log_int(rng, 1, max(1, 1024 * 128 * 128 // (H * d[0] * d[1])))
        return dict(op=op, dtype=dtype, B=B, H=H, dk=d[0], dv=d[1], decay=rng.choice(("token", "head")))
    d = rng.choice((32, 64, 128, 256)) if rng.random() < 0.7 else rng.randint(1, 256)
    H = rng.choice((1, 3, 4, 8, 16, 24))
    B = rng.choice((1, 2, 4, 7))
    L = _log_int(rng, 1, max(1, (1 << 25) // (B * H * d)))
    c = dict(op=op, dtype=dtype, B=B, L=L, H=H, d=d, weight=rng.random() < 0.7, fused=rng.randint(1, 3), train=rng.random() < 0.6)
    if op == "hnorm":
        return dict(c, kind=rng.choice(("l2", "rms")))
    return dict(c, act=rng.choice(("silu", "sigmoid")), residual=rng.random() < 0.5)


def _dt(case):
    return torch.float32 if case["dtype"] == "fp32" else torch.bfloat16


def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] in ("fwd", "bwd"):
        BH, L, dk, dv = case["B"] * case["H"], case["L"], case["dk"], case["dv"]
        g = BH * L * e if case["decay"] == "token" else case["H"] * 4
        S = BH * dk * dv * 4
        if case["op"] == "fwd":
            return {"bytes": BH * L * 2 * (dk + dv) * e + g + S * (2 if case["s0"] else 1), "flops": 4 * BH * L * dk * dv}
        n = BH * L * (4 * dk + 3 * dv) * e + g * (2 if case["decay"] == "token" else 1)
        return {"bytes": n + S * (3 if case["s0"] else 0), "flops": 10 * BH * L * dk * dv}
    if case["op"] == "step":
        BH, dk, dv = case["B"] * case["H"], case["dk"], case["dv"]
        return {"bytes": BH * (2 * dk * dv * 4 + 2 * (dk + dv) * e), "flops": 4 * BH * dk * dv}
    n, d = case["B"] * case["L"] * case["H"], case["d"]
    if case["op"] == "hnorm":
        return {"bytes": n * d * e * (5 if case["train"] else 2), "flops": n * d * (12 if case["train"] else 4)}
    tensors = 3 + (1 if case["residual"] else 0) + (5 if case["train"] else 0)
    return {"bytes": n * d * e * tensors, "flops": n * d * (30 if case["train"] else 10)}


# ---------------------------------------------------------------------------------------------- inputs
def _log_decay(case, g, shape):
    """Token form: log sigmoid of a per-head level plus noise, so that heads remember from about 3 to about 1000 tokens;
    the first token of a later document forgets everything.  Head form: 1 - 2^-x, evenly spaced in x."""
    H = case["H"]
    if case["decay"] == "head":
        x = torch.linspace(1.5, 11.0, H, device=DEV) + 0.3 * torch.rand(H, generator=g, device=DEV)
        return torch.log1p(-torch.exp2(-x))
    level = 1.0 + 6.0 * torch.rand((1, H) + (1,) * (len(shape) - 2), generator=g, device=DEV)
    l = torch.nn.functional.logsigmoid(level + torch.randn(shape, generator=g, device=DEV))
    if case.get("docs") and case["L"] > 1:
        B, L = case["B"], case["L"]
        at = torch.randint(1, L, (B, case["docs"]), generator=g, device=DEV)
        l = l.masked_fill(torch.zeros(B, L, dtype=torch.bool, device=DEV).scatter_(1, at, True)[:, None, :], float("-inf"))
    return l.to(_dt(case))


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = _dt(case)

    def n(*shape, std=1.0, dtype=dt):
        return (std * torch.randn(shape, generator=g, device=DEV)).to(dtype)

    s = dict(case=case)
    if case["op"] in ("fwd", "bwd", "step"):
        B, H, dk, dv = case["B"], case["H"], case["dk"], case["dv"]
        t = () if case["op"] == "step" else (case["L"],)
        s["q"], s["k"] = n(B, H, *t, dk, std=dk ** -0.5), n(B, H, *t, dk, std=dk ** -0.5)
        s["v"] = n(B, H, *t, dv)
        s["l"] = _log_decay(case, g, (B, H) + t)
        if case["op"] == "step":
            s["S"] = n(B, H, dk, dv, std=0.3, dtype=torch.float32)
            return s
        s["S0"] = n(B, H, dk, dv, std=0.3, dtype=torch.float32) if case["s0"] else None
        if case["op"] == "bwd":
            s["dO"] = n(B, H, *t, dv)
            s["dS"] = n(B, H, dk, dv, std=0.1, dtype=torch.float32) if case["s0"] else None
        return s
    B, L, H, d, f = case["B"], case["L"], case["H"], case["d"], case["fused"]
    proj = n(B, L, f, H, d)  # one fused projection; the operator reads a slice of it
    s["w"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)) if case["weight"] else None
    if case["op"] == "hnorm":
        s["x"], s["dy"] = proj[:, :, 0], n(B, H, L, d)
        return s
    s["o"], s["gate"], s["dy"] = n(B, H, L, d, std=1.5), proj[:, :, f - 1], n(B, L, H, d)
    s["residual"] = n(B, L, H, d) if case["residual"] else None
    return s


# ---------------------------------------------------------------------------------------------- plain forms
def _walk(x, y, z, l, S0, C=128):
    """o_t = sum_{s<=t} e^{l_{s+1}+..+l_t} (x_t.y_s) z_s + e^{l_1+..+l_t} S0^T x_t and the state after the last token, by
    chunks of C tokens: float32, with the sums of log-decays in 64 bits.  l: [B,H,L] float64, finite."""
    B, H, L, a = x.shape
    b = z.shape[-1]
    C = min(C, max(1, L))
    N = -(-L // C)
    pad = N * C - L

    def cut(t):
        return torch.nn.functional.pad(t, (0, 0, 0, pad)).view(B, H, N, C, t.shape[-1])

    x, y, z = cut(x), cut(y), cut(z)
    c = torch.nn.functional.pad(l, (0, pad)).view(B, H, N, C).cumsum(-1)
    D = torch.exp((c[..., :, None] - c[..., None, :]).masked_fill(
        torch.ones(C, C, dtype=torch.bool, device=x.device).triu(1), -math.inf)).float()
    intra = ((x @ y.transpose(-1, -2)) * D) @ z
    del D
    add = (y * torch.exp(c[..., -1:] - c).float()[..., None]).transpose(-1, -2) @ z  # [B,H,N,a,b]
    T = c[..., -1].cumsum(-1)  # the log-decay up to the end of every chunk
    T0 = torch.nn.functional.pad(T, (1, 0))
    E = torch.exp((T0[..., :, None] - T0[..., None, 1:]).masked_fill(
        torch.ones(N + 1, N, dtype=torch.bool, device=x.device).triu(0), -math.inf)).float()  # state before chunk n <- chunk m
    S = (E @ add.reshape(B, H, N, a * b)).view(B, H, N + 1, a, b)
    if S0 is not None:
        S = S + torch.exp(T0).float()[..., None, None] * S0[:, :, None]
    o = intra + torch.exp(c).float()[..., None] * (x @ S[:, :, :N])
    return o.reshape(B, H, N * C, b)[:, :, :L], S[:, :, N]


def _l64(s, L):
    l = s["l"].double()
    if l.dim() == 1:
        l = l[None, :, None].expand(s["case"]["B"], -1, L)
    return l.clamp_min(-1e3)  # e^-1000 is 0 in float32 and leaves 64-bit sums exact enough


def _plain_attention(s):
    case = s["case"]
    dt, L = _dt(case), case["L"]
    q, k, v, S0, l = s["q"].float(), s["k"].float(), s["v"].float(), s["S0"], _l64(s, case["L"])
    if case["op"] == "fwd":
        o, S = _walk(q, k, v, l, S0)
        return o.to(dt), S
    dO, dS = s["dO"].float(), s["dS"]
    # reversed in time the decay that leads from a token to the one before it is its own; the first one's leads to S0
    lr = torch.nn.functional.pad(l, (0, 1))[..., 1:].flip(-1)
    dq, St = _walk(dO, v, k, l, None if S0 is None else S0.transpose(-1, -2).contiguous())
    dk, _ = _walk(v.flip(2), dO.flip(2), q.flip(2), lr, None if dS is None else dS.transpose(-1, -2).contiguous())
    dv, G = _walk(k.flip(2), q.flip(2), dO.flip(2), lr, dS)
    dk, dv = dk.flip(2), dv.flip(2)
    out = [dq.to(dt), dk.to(dt), dv.to(dt)]
    if case["decay"] == "token":
        m = ((q * dq).sum(-1, dtype=torch.float64) - (k * dk).sum(-1, dtype=torch.float64)).flip(-1).cumsum(-1).flip(-1)
        if dS is not None:
            m = m + (dS.double() * St.transpose(-1, -2).double()).sum((-1, -2))[..., None]
        out.append(m.to(dt))
    if S0 is not None:
        out.append(torch.exp(l[..., 0]).float()[..., None, None] * G)
    return out


def _plain_step(s):
    case = s["case"]
    q, k, v, l, S = s["q"].float(), s["k"].float(), s["v"].float(), s["l"].float(), s["S"]
    g = torch.exp(l)
    g = g[None, :, None, None] if g.dim() == 1 else g[..., None, None]
    S.copy_(g * S + k[..., :, None] * v[..., None, :])
    return (q[..., None, :] @ S)[..., 0, :].to(_dt(case)), S


def _plain_hnorm(s):
    case = s["case"]
    dt, d = _dt(case), case["d"]
    x, scale, m = s["x"].float(), _scale(case), 1.0 if case["kind"] == "l2" else 1.0 / case["d"]
    w = 1.0 if s["w"] is None else s["w"]
    r = torch.rsqrt((x * x).sum(-1, keepdim=True) * m + EPS)
    y = (scale * (x * r) * w).transpose(1, 2).contiguous().to(dt)
    if not case["train"]:
        return y
    dy = s["dy"].transpose(1, 2).float()
    dn = scale * dy * w
    dx = r * (dn - m * (x * r) * (dn * (x * r)).sum(-1, keepdim=True))
    return [y, dx.to(dt)] + ([] if s["w"] is None else [(scale * dy * (x * r)).reshape(-1, d).sum(0)])


def _plain_gnorm(s):
    case = s["case"]
    dt, d, scale = _dt(case), case["d"], _scale(case)
    o, gate = s["o"].transpose(1, 2).float(), s["gate"].float()
    w = 1.0 if s["w"] is None else s["w"]
    sg = torch.sigmoid(gate)
    a = gate * sg if case["act"] == "silu" else sg
    r = torch.rsqrt((o * o).sum(-1, keepdim=True) / d + EPS)
    y = scale * (o * r) * w * a
    if s["residual"] is not None:
        y = y + s["residual"].float()
    if not case["train"]:
        return y.to(dt)
    dy = s["dy"].float()
    da = sg * (1 + gate * (1 - sg)) if case["act"] == "silu" else sg * (1 - sg)
    dn = scale * dy * w * a
    do = r * (dn - (o * r) * (dn * (o * r)).sum(-1, keepdim=True) / d)
    out = [y.to(dt), do.transpose(1, 2).contiguous().to(dt), (scale * dy * (o * r) * w * da).to(dt)]
    return out + ([] if s["w"] is None else [(scale * dy * (o * r) * a).reshape(-1, d).sum(0)])


def _scale(case):
    return case["d"] ** -0.5 if case["op"] == "hnorm" and case["kind"] == "rms" else 0.75


# ---------------------------------------------------------------------------------------------- one pass
def _own(s):
    from delta_rule_linear_efla_b200 import decay, norms

    case, op = s["case"], s["case"]["op"]
    dt = _dt(case)
    if op == "fwd":
        return decay.decay_chunk_fwd(s["q"], s["k"], s["v"], s["l"], s["S0"], o_dtype=dt)
    if op == "bwd":
        r = decay.decay_bwd(s["q"], s["k"], s["v"], s["l"], s["dO"], s["S0"], s["dS"], want_dS0=s["S0"] is not None)
        return [t for t in r if t is not None]
    if op == "step":
        return decay.decay_recurrent_step(s["q"], s["k"], s["v"], s["l"], s["S"], o_dtype=dt), s["S"]
    scale = _scale(case)
    if op == "hnorm":
        a = dict(weight=s["w"], kind=case["kind"], scale=scale, eps=EPS)
        y = norms.head_norm_fwd(s["x"], **a)
        return [t for t in (y, *norms.head_norm_bwd(s["x"], s["dy"], **a)) if t is not None] if case["train"] else y
    a = dict(weight=s["w"], scale=scale, eps=EPS, act=case["act"])
    y = norms.gated_norm_fwd(s["o"], s["gate"], residual=s["residual"], **a)
    return [t for t in (y, *norms.gated_norm_bwd(s["o"], s["gate"], s["dy"], **a)) if t is not None] if case["train"] else y


def run(s):
    if own:
        return _own(s)
    return {"fwd": _plain_attention, "bwd": _plain_attention, "step": _plain_step, "hnorm": _plain_hnorm,
            "gnorm": _plain_gnorm}[s["case"]["op"]](s)


# ---------------------------------------------------------------------------------------------- exact values
def _recurrence(x, y, z, decay, S, after=False):
    """The definition, token by token in 64 bits: S <- decay_t S + y_t z_t^T, o_t = S^T x_t (tensors [BH,L,.]).
    after: the decay of a token is applied once it has been read (time running backwards)."""
    o = torch.empty(x.shape[0], x.shape[1], z.shape[2], dtype=torch.float64, device=x.device)
    for t in (range(x.shape[1] - 1, -1, -1) if after else range(x.shape[1])):
        if not after:
            S.mul_(decay[:, t, None, None])
        S.baddbmm_(y[:, t, :, None], z[:, t, None, :])
        torch.bmm(x[:, t, None, :], S, out=o[:, t : t + 1])
        if after:
            S.mul_(decay[:, t, None, None])
    return o, S


def exact(case, seed):
    s = prepare(case, seed)
    f = {n: t.double() for n, t in s.items() if isinstance(t, torch.Tensor)}
    op = case["op"]
    if op in ("fwd", "bwd", "step"):
        B, H, dk, dv, L = case["B"], case["H"], case["dk"], case["dv"], case.get("L", 1)
        g = torch.exp(f["l"])
        g = (g[None, :, None].expand(B, H, L) if g.dim() == 1 else g).reshape(B * H, L)

        def flat(n, d):
            return f[n].reshape(B * H, L, d)

        def state(n):
            return f[n].reshape(B * H, dk, dv).clone() if n in f else torch.zeros(B * H, dk, dv, dtype=torch.float64, device=DEV)

        q, k, v = flat("q", dk), flat("k", dk), flat("v", dv)
        if op != "bwd":
            o, S = _recurrence(q, k, v, g, state("S0" if op == "fwd" else "S"))
            return o.view(*s["v"].shape), S.view(B, H, dk, dv)
        dO = flat("dO", dv)
        dq, St = _recurrence(dO, v, k, g, state("S0").transpose(1, 2).contiguous())
        dk_, _ = _recurrence(v, dO, q, g, state("dS").transpose(1, 2).contiguous(), after=True)
        dv_, G = _recurrence(k, q, dO, g, state("dS"), after=True)
        out = [dq.view(B, H, L, dk), dk_.view(B, H, L, dk), dv_.view(B, H, L, dv)]
        if case["decay"] == "token":
            # d/dl_t = e^{l_t} <dL/dS_t, S_{t-1}>, which telescopes from the sequence's end
            tail = (St.transpose(1, 2) * state("dS")).sum((1, 2))
            m = (q * dq).sum(-1) - (k * dk_).sum(-1)
            out.append((m.flip(1).cumsum(1).flip(1) + tail[:, None]).view(B, H, L))
        return out + ([G.view(B, H, dk, dv)] if case["s0"] else [])
    d, scale = case["d"], _scale(case)
    w = f.get("w", torch.ones(d, dtype=torch.float64, device=DEV)).clone().requires_grad_(True)
    if op == "hnorm":
        x = f["x"].requires_grad_(True)
        norm = x.square().sum(-1, keepdim=True) if case["kind"] == "l2" else x.square().mean(-1, keepdim=True)
        y = (scale * w * x / (norm + EPS).sqrt()).transpose(1, 2)
        leaves = [x, w]
    else:
        o, gate = f["o"].requires_grad_(True), f["gate"].requires_grad_(True)
        a = torch.sigmoid(gate) * (gate if case["act"] == "silu" else 1)
        t = o.transpose(1, 2)
        y = scale * a * w * t / (t.square().mean(-1, keepdim=True) + EPS).sqrt()
        y = y + f["residual"] if "residual" in f else y
        leaves = [o, gate, w]
    if not case["train"]:
        return y.detach()
    grads = torch.autograd.grad(y, leaves, f["dy"])
    return [y.detach(), *(grads if "w" in f else grads[:-1])]
