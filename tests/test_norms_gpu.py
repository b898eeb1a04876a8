"""The per-head norms on the GPU against their formulas in 64 bits.

Tolerances in half steps u (bf16 2^-8, fp32 2^-24): the arithmetic is fp32, a row's sum of d <= 256 squares is
off by at most a few u (lanes add eight or fewer in turn, then pairwise), so outputs are within u of their type
plus 32 fp32 half steps; the weight's gradient adds rows in turn (up to a few hundred a thread) and then
pairwise: 256 fp32 half steps of the 2-norm."""
import pytest
import torch

import decay_ref as R
from delta_rule_linear_efla_b200 import efla, norms

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def near(x, ref, dtype, extra=32):
    rel, big = R.far(x, ref)
    tol = U[dtype] + extra * 2.0 ** -24
    assert rel <= tol and big <= 8 * tol, (rel, big, tol)


def rnd(*shape, dtype, seed, std=1.0):
    return (std * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


def views(x):
    """The same [B,L,H,d] values dense, as a slice of a fused projection, off alignment, and head-major."""
    B, L, H, d = x.shape
    fused = torch.zeros(B, L, 3, H, d, dtype=x.dtype, device="cuda")
    fused[:, :, 1] = x
    odd = torch.zeros(x.numel() + 1, dtype=x.dtype, device="cuda")
    odd[1:] = x.reshape(-1)
    return {"dense": x, "fused": fused[:, :, 1], "odd": odd[1:].view(x.shape),
            "heads": x.transpose(1, 2).contiguous().transpose(1, 2)}


SHAPES = [(2, 5, 3, 128), (1, 1, 1, 64), (2, 33, 4, 80), (1, 7, 2, 256), (3, 4, 5, 1), (1, 9, 3, 33), (2, 3, 2, 200),
          (1, 600, 16, 128), (1, 3, 2, 8)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["l2", "rms"])
@pytest.mark.parametrize("w_dtype", [None, F32, BF])
@pytest.mark.parametrize("shape", SHAPES)
def test_head_norm(shape, w_dtype, kind, dtype):
    B, L, H, d = shape
    x = rnd(*shape, dtype=dtype, seed=1, std=2.0)
    w = None if w_dtype is None else rnd(d, dtype=w_dtype, seed=2)
    dy = rnd(B, H, L, d, dtype=dtype, seed=3)
    xr = x.double().requires_grad_(True)
    wr = None if w is None else w.double().requires_grad_(True)
    ref = R.head_norm(xr, wr, kind, 0.5, 1e-5)
    grads = torch.autograd.grad(ref, [xr] + ([] if w is None else [wr]), dy.double())
    for how, v in views(x).items():
        y = norms.head_norm_fwd(v, w, kind, 0.5, 1e-5)
        assert y.is_contiguous() and y.shape == (B, H, L, d)
        near(y, ref, dtype)
        dx, dw = norms.head_norm_bwd(v, dy, w, kind, 0.5, 1e-5)
        # dx is a difference that can cancel (d = 1 leaves only eps): against the size of its parts
        part = (dy.double().transpose(1, 2) * (1 if w is None else w.double())).norm() * 0.5
        size = part / x.double().square().sum(-1).mean().sqrt().clamp_min(1e-3) * (d ** 0.5 if kind == "rms" else 1)
        tol = U[dtype] * grads[0].norm() + 64 * 2.0 ** -24 * size
        assert (dx.double() - grads[0]).norm() <= tol, how
        if w is None:
            assert dw is None
        else:
            assert dw.dtype == w.dtype
            near(dw, grads[1], w.dtype, 256)


@pytest.mark.parametrize("dtype,o_dtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("w_dtype,res", [(None, False), (F32, True), (BF, True)])
@pytest.mark.parametrize("shape", SHAPES)
def test_gated_norm(shape, w_dtype, res, act, dtype, o_dtype):
    B, L, H, d = shape
    o = rnd(B, H, L, d, dtype=o_dtype, seed=1, std=2.0)
    gate = rnd(*shape, dtype=dtype, seed=2, std=3.0)
    w = None if w_dtype is None else rnd(d, dtype=w_dtype, seed=3)
    r = rnd(*shape, dtype=dtype, seed=4) if res else None
    dy = rnd(*shape, dtype=dtype, seed=5)
    leaves = [o.double().requires_grad_(True), gate.double().requires_grad_(True)]
    wr = None if w is None else w.double().requires_grad_(True)
    ref = R.gated_norm(*leaves, wr, r, 1.5, 1e-5, act)
    grads = torch.autograd.grad(ref, leaves + ([] if w is None else [wr]), dy.double())
    rv = views(r) if res else None
    for how, v in views(gate).items():
        y = norms.gated_norm_fwd(o, v, w, rv[how] if res else None, 1.5, 1e-5, act)
        near(y, ref, dtype)
        do, dg, dw = norms.gated_norm_bwd(o, v, dy, w, 1.5, 1e-5, act)
        part = (dy.double() * gate.double().sigmoid() * (gate.double() if act == "silu" else 1) *
                (1 if w is None else w.double())).norm() * 1.5
        tol = U[o_dtype] * grads[0].norm() + 64 * 2.0 ** -24 * part / o.double().square().mean(-1).sqrt().mean().clamp_min(1e-3)
        assert do.dtype == o_dtype and (do.double() - grads[0]).norm() <= tol, how
        near(dg, grads[1], dtype)
        if w is not None:
            near(dw, grads[2], w.dtype, 256)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_extremes(dtype):
    """Rows of zeros, large gates of both signs, rows of one value: finite, and the formula's."""
    o = torch.zeros(1, 1, 4, 64, dtype=dtype, device="cuda")
    o[0, 0, 1], o[0, 0, 2], o[0, 0, 3] = 1.0, 1e4, -1e-4
    gate = torch.tensor([-100.0, 100.0, 0.0, -1000.0], device="cuda")[None, :, None, None].expand(1, 4, 1, 64).to(dtype).contiguous()
    y = norms.gated_norm_fwd(o, gate)
    near(y, R.gated_norm(o, gate, None, None, 1.0, 1e-6, "silu"), dtype)
    grads = norms.gated_norm_bwd(o, gate, torch.ones_like(gate))
    assert all(torch.isfinite(g).all() for g in grads if g is not None)
    x = torch.zeros(1, 2, 1, 64, dtype=dtype, device="cuda")
    assert not norms.head_norm_fwd(x).any() and torch.isfinite(norms.head_norm_bwd(x, torch.ones(1, 1, 2, 64, dtype=dtype, device="cuda"))[0]).all()


def test_no_rows():
    w = torch.ones(64, device="cuda")
    x = torch.empty(2, 0, 3, 64, device="cuda")
    assert norms.head_norm_fwd(x, w).shape == (2, 3, 0, 64)
    dx, dw = norms.head_norm_bwd(x, torch.empty(2, 3, 0, 64, device="cuda"), w)
    assert dx.shape == x.shape and not dw.any()
    _, _, dw = norms.gated_norm_bwd(torch.empty(2, 3, 0, 64, device="cuda"), x, x, w)
    assert not dw.any()


def test_residual_in_place_and_repeatable():
    o, gate, r = rnd(1, 4, 300, 128, dtype=BF, seed=1), rnd(1, 300, 4, 128, dtype=BF, seed=2), rnd(1, 300, 4, 128, dtype=BF, seed=3)
    w = rnd(128, dtype=F32, seed=4)
    ref = norms.gated_norm_fwd(o, gate, w, r)
    a, b = (norms.gated_norm_bwd(o, gate, r, w) for _ in range(2))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    y = norms.gated_norm_fwd(o, gate, w, r, y=r)
    assert y is r and torch.equal(y, ref)


def test_broadcast_gate_and_residual():
    """Views whose tokens or heads are one and the same (strides of zero)."""
    o = rnd(2, 4, 50, 128, dtype=BF, seed=1)
    gate = rnd(2, 50, 1, 128, dtype=BF, seed=2).expand(2, 50, 4, 128)
    res = rnd(1, 1, 4, 128, dtype=BF, seed=3).expand(2, 50, 4, 128)
    near(norms.gated_norm_fwd(o, gate, None, res), R.gated_norm(o, gate, None, res, 1.0, 1e-6, "silu"), BF)
    dy = rnd(2, 50, 4, 128, dtype=BF, seed=4)
    a, b = norms.gated_norm_bwd(o, gate, dy), norms.gated_norm_bwd(o, gate.contiguous(), dy)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_another_stream():
    o, gate = rnd(1, 4, 500, 128, dtype=BF, seed=1), rnd(1, 500, 4, 128, dtype=BF, seed=2)
    ref = norms.gated_norm_fwd(o, gate)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = norms.gated_norm_fwd(o, gate, stream=s)
    s.synchronize()
    assert torch.equal(y, ref)


def test_autograd_and_capture():
    x, w = rnd(1, 40, 2, 64, dtype=BF, seed=1).requires_grad_(True), rnd(64, dtype=F32, seed=2).requires_grad_(True)
    dy = rnd(1, 2, 40, 64, dtype=BF, seed=3)
    norms.head_norm(x, w, "rms", 2.0).backward(dy)
    dx, dw = norms.head_norm_bwd(x.detach(), dy, w.detach(), "rms", 2.0)
    assert torch.equal(x.grad, dx) and torch.equal(w.grad, dw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        norms.head_norm_bwd(x.detach(), dy, w.detach())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = norms.head_norm_bwd(x.detach(), dy, w.detach(), "rms", 2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], dx) and torch.equal(got[1], dw)


@pytest.mark.parametrize("attention", ["decay", "efla"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_between_its_norms(attention, dtype):
    """The whole run as a layer uses it: q and k out of one projection, normalised; the attention; its
    readout normalised, gated, scaled and added to the residual; gradients to every input.  Against the
    composition of the formulas in 64 bits: five roundings to the type on the way (q, k, o, y and, in the
    gradients, the same again)."""
    from delta_rule_linear_efla_b200 import decay

    B, L, H, d = 2, 130, 2, 64
    proj = rnd(B, L, 3, H, d, dtype=dtype, seed=1).requires_grad_(True)
    gate, res = (rnd(B, L, H, d, dtype=dtype, seed=s).requires_grad_(True) for s in (2, 3))
    w = rnd(d, dtype=F32, seed=4).requires_grad_(True)
    aux = rnd(B, H, L, dtype=F32, seed=5)
    aux = (torch.nn.functional.logsigmoid(3 + aux) if attention == "decay" else torch.sigmoid(aux)).to(dtype).requires_grad_(True)
    dy = rnd(B, L, H, d, dtype=dtype, seed=6)
    leaves = [proj, gate, res, w, aux]
    q, k, v = (t.transpose(1, 2) for t in proj.unbind(2))
    call = decay.decay_attention if attention == "decay" else efla.efla_attention
    y, _ = call(q.contiguous(), k.contiguous(), v.contiguous(), aux, qk_norm="l2", gate=gate, norm_weight=w, residual=res,
                scale=0.5)
    got = torch.autograd.grad(y, leaves, dy)

    ref_leaves = [t.detach().double().requires_grad_(True) for t in leaves]
    pr, gr, rr, wr, ar = ref_leaves
    qr, kr = (R.head_norm(pr[:, :, i], None, "l2", 1.0, 1e-6) for i in (0, 1))
    vr = pr[:, :, 2].transpose(1, 2)
    if attention == "decay":
        o, _ = R.recurrence(qr, kr, vr, ar)
    else:
        S, o = torch.zeros(B, H, d, d, dtype=torch.float64, device="cuda"), []
        for t in range(L):
            lam = kr[:, :, t].square().sum(-1)
            al = (-torch.expm1(-ar[:, :, t] * lam) / lam)[..., None, None]
            S = S + al * kr[:, :, t, :, None] * (vr[:, :, t, None, :] - kr[:, :, t, None, :] @ S)
            o.append((qr[:, :, t, None, :] @ S)[:, :, 0])
        o = torch.stack(o, 2)
    yr = R.gated_norm(o, gr, wr, rr, 0.5, 1e-6, "silu")
    ref = torch.autograd.grad(yr, ref_leaves, dy.double())
    tol = 5 * U[dtype] + 256 * 2.0 ** -24
    assert R.far(y, yr)[0] <= tol
    for n, a, b in zip(("proj", "gate", "residual", "weight", "aux"), got, ref):
        assert R.far(a, b)[0] <= 2 * tol, (n, R.far(a, b))
