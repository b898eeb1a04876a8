"""Refusals of the decayed attention's and the norms' entry points, on the host before any CUDA call (the
fake addresses are never dereferenced on these paths), and the plain reference forms that the GPU tests use,
pinned against differences."""
import ctypes
import math

import pytest
import torch

import decay_ref as R
from delta_rule_linear_efla_b200 import decay, efla, norms

P = 0x10000
F32, BF16 = efla.EFLA_F32, efla.EFLA_BF16
NULL, SHAPE, DTYPE, UNSUPPORTED, WORKSPACE, ALIGN, OPTION = 1, 2, 3, 4, 7, 8, 11


@pytest.fixture(scope="module")
def lib():
    from delta_rule_linear_efla_b200 import build

    build.build()
    return efla.load_library()


def fwd(lib, **kw):
    a = dict(q=P, k=P, v=P, g=P, form=0, S0=None, o=P, Sf=P, B=1, H=1, L=64, dk=64, dv=64, dt=BF16, odt=BF16, ws=None, n=0)
    a.update(kw)
    return lib.efla_decay_chunk_fwd(*[a[x] for x in "q k v g form S0 o Sf B H L dk dv dt odt ws n".split()], None)


def bwd(lib, **kw):
    a = dict(q=P, k=P, v=P, g=P, form=0, S0=None, dO=P, dS=None, dq=P, dk_=P, dv_=P, dl=P, dS0=None, B=1, H=1, L=64, dk=64,
             dv=64, dt=F32, ws=P, n=0)
    a.update(kw)
    return lib.efla_decay_bwd(*[a[x] for x in "q k v g form S0 dO dS dq dk_ dv_ dl dS0 B H L dk dv dt ws n".split()], None)


def step(lib, **kw):
    a = dict(q=P, k=P, v=P, g=P, form=0, S=P, o=P, B=1, H=1, dk=64, dv=64, dt=BF16, odt=BF16)
    a.update(kw)
    return lib.efla_decay_recurrent_step(*[a[x] for x in "q k v g form S o B H dk dv dt odt".split()], None)


SHARED = [(dict(dt=5), DTYPE), (dict(form=2), OPTION), (dict(B=0), SHAPE), (dict(H=-1), SHAPE), (dict(dk=0), SHAPE),
          (dict(B=1 << 13, H=1 << 12), SHAPE), (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL),
          (dict(g=None), NULL), (dict(k=P + 1), ALIGN), (dict(g=P + 1), ALIGN)]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(odt=3), DTYPE), (dict(L=-1), SHAPE), (dict(L=0x7fffffff), SHAPE), (dict(dk=129), UNSUPPORTED), (dict(o=None), NULL),
    (dict(S0=P + 2), ALIGN), (dict(Sf=P + 2), ALIGN), (dict(o=P + 1), ALIGN), (dict(form=1, g=P + 2), ALIGN),
    (dict(L=4096), WORKSPACE), (dict(L=4096, ws=P, n=64), WORKSPACE), (dict(L=4096, ws=P + 8, n=1 << 40), ALIGN)])
def test_forward_refusals(lib, kw, status):
    assert fwd(lib, **kw) == status


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(form=1), OPTION), (dict(L=-1), SHAPE), (dict(dv=130), UNSUPPORTED), (dict(dO=None), NULL), (dict(dq=None), NULL),
    (dict(dv_=None), NULL), (dict(dl=P + 2), ALIGN), (dict(dS=P + 1), ALIGN), (dict(dS0=P + 1), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(n=16), WORKSPACE), (dict(ws=P + 4, n=1 << 40), ALIGN)])
def test_backward_refusals(lib, kw, status):
    assert bwd(lib, **kw) == status


@pytest.mark.parametrize("kw,status", SHARED + [(dict(dk=257), UNSUPPORTED), (dict(S=None), NULL), (dict(S=P + 8), ALIGN),
                                                (dict(o=None), NULL), (dict(odt=9), DTYPE)])
def test_step_refusals(lib, kw, status):
    assert step(lib, **kw) == status


def test_workspace_sizes(lib):
    f, b = lib.efla_decay_chunk_fwd_workspace_size, lib.efla_decay_bwd_workspace_size
    for bad in ((0, 1, 64, 64, 64, BF16), (1, 1, 64, 129, 64, BF16), (1, 1, 64, 64, 64, 7), (1, 1, 0, 64, 64, BF16)):
        assert f(*bad) == 0 and b(*bad) == 0
    assert b(1, 1, 64, 64, 64, F32) > 0
    assert f(1, 1, 64, 64, 64, BF16) == 0  # one chunk: nothing to cut


def norm(lib, which, **kw):
    st = (ctypes.c_longlong * 3)(64, 64, 64)
    a = dict(x=P, st=st, odt=F32, w=P, wdt=F32, res=None, rst=None, dy=P, y=P, y2=P, dw=P, B=1, L=1, H=1, d=64, dt=BF16, opt=0,
             scale=1.0, eps=1e-6, ws=P, n=1 << 30)
    a.update(kw)
    order = {"head": "x st w wdt y B L H d dt opt scale eps", "head_bwd": "x st w wdt dy y dw B L H d dt opt scale eps ws n",
             "gated": "x odt y2 st w wdt res rst y B L H d dt opt scale eps",
             "gated_bwd": "x odt y2 st w wdt dy y x dw B L H d dt opt scale eps ws n"}[which]
    entry = {"head": lib.efla_head_norm, "head_bwd": lib.efla_head_norm_bwd, "gated": lib.efla_gated_norm,
             "gated_bwd": lib.efla_gated_norm_bwd}[which]
    return entry(*[a[x] for x in order.split()], None)


@pytest.mark.parametrize("which", ["head", "head_bwd", "gated", "gated_bwd"])
@pytest.mark.parametrize("kw,status", [
    (dict(dt=4), DTYPE), (dict(wdt=4), DTYPE), (dict(opt=2), OPTION), (dict(eps=-1.0), OPTION), (dict(eps=math.nan), OPTION),
    (dict(eps=math.inf), OPTION), (dict(scale=math.nan), OPTION), (dict(B=-1), SHAPE), (dict(d=0), SHAPE),
    (dict(d=257), UNSUPPORTED), (dict(x=None), NULL), (dict(y=None), NULL), (dict(st=None), NULL), (dict(w=P + 2), ALIGN),
    (dict(y=P + 1), ALIGN), (dict(B=1 << 20, L=1 << 20, H=1 << 20), SHAPE)])
def test_norm_refusals(lib, which, kw, status):
    assert norm(lib, which, **kw) == status


def test_norm_backward_refusals(lib):
    for which in ("head_bwd", "gated_bwd"):
        assert norm(lib, which, dy=None) == NULL
        assert norm(lib, which, w=None) == NULL  # a gradient of no weight
        assert norm(lib, which, ws=None) == WORKSPACE
        assert norm(lib, which, n=64) == WORKSPACE
        assert norm(lib, which, ws=P + 8) == ALIGN
    assert norm(lib, "gated", res=P) == NULL  # a residual without strides
    assert norm(lib, "gated", odt=7) == DTYPE
    assert lib.efla_norm_bwd_workspace_size(0) == 0 and lib.efla_norm_bwd_workspace_size(257) == 0
    assert "option" in efla.status_str(OPTION)


def test_binding_refusals_without_a_device():
    q = torch.zeros(1, 1, 4, 16)
    for call in (lambda: decay.decay_chunk_fwd(q, q, q, q[..., 0]), lambda: decay.decay_bwd(q, q, q, q[..., 0], q),
                 lambda: decay.decay_recurrent_step(q[0], q[0], q[0], q[0, ..., 0], q), lambda: norms.head_norm_fwd(q),
                 lambda: norms.gated_norm_fwd(q, q), lambda: decay.decay_attention(q, q, q, q[..., 0])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="no gradient"):
        decay.decay_attention(q, q, q, torch.zeros(1, requires_grad=True))
    with pytest.raises(ValueError, match="gate"):
        efla.efla_attention(q, q, q, q[..., 0], scale=0.5)


def test_reference_gradients_against_differences():
    """The references' own autograd against central differences in 64 bits (truncation h^2 ~ 1e-10)."""
    g = torch.Generator().manual_seed(1)

    def n(*s):
        return torch.randn(s, generator=g, dtype=torch.float64)

    x = [n(1, 2, 6, 3), n(1, 2, 6, 3), n(1, 2, 6, 4), -n(1, 2, 6).abs(), n(1, 2, 3, 4)]
    dO, dS = n(1, 2, 6, 4), n(1, 2, 3, 4)
    grads = R.gradients(*x, dO, dS)
    f = lambda y: (lambda o, S: float((o * dO).sum() + (S * dS).sum()))(*R.recurrence(*y))  # noqa: E731
    for i in range(5):
        d = n(*x[i].shape)
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + 1e-5 * d, x[i] - 1e-5 * d
        assert abs((f(up) - f(down)) / 2e-5 - float((grads[i] * d).sum())) <= 1e-7
