"""Gradients of the decayed attention over rows of several documents, over long rows and past 32-bit offsets,
against the token recurrence in 64 bits (walked in both directions, without autograd, so that rows can be long).

Tolerances, in half steps u (bf16 2^-8, fp32 2^-24) of the 2-norm; an element may be off by eight times that of
max(rms, |value|).  dq, dk, dv, dS0 and the fp32 log-decay's gradient: as in the tests of single rows.  The bf16
gradient of the log-decay has two roundings to the type: its own, and one of each product (v_s . dO_t) that straddles
the token (the others cancel, dq and dk round the same products).  The rms of a rounding is at most u / sqrt(3) of its
value, and independent ones add up like the values do: sqrt(2/3) u of the rms, below u.  What the fp32 sums of dots
and the two halves of the states' copies add in a row of L tokens is at most 2^-17 sqrt(L) of the dots: 2^-9 for
65536, in quadrature sqrt(2/3 + 1/4) u, still below u."""
import pytest
import torch

from decay_walked_ref import walked_gradients
from delta_rule_linear_efla_b200 import decay, efla
from test_decay_gpu import BF, F32, OUT, STATE, make, near

pytestmark = pytest.mark.gpu

DL = {BF: 2.0 ** -8, F32: 4 * OUT[F32]}
INF = float("inf")


def check(x, dO, dS, got, level=1):
    """Every gradient; a log-decay of -inf has exactly none.  level: of the state's tolerance."""
    ref = walked_gradients(*x, dO, dS)
    dtype = x[0].dtype
    for a, b in zip(got[:3], ref[:3]):
        near(a, b, OUT[dtype])
    if got[3] is not None:
        assert not got[3][torch.isinf(x[3])].any()
        near(got[3], ref[3], DL[dtype])
    if got[4] is not None:
        near(got[4], ref[4], level * STATE[dtype])
    assert efla.last_device_error() == 0


def documents(x, starts):
    x[3][:, :, starts] = -INF
    return list(zip([0] + starts, starts + [x[0].shape[2]]))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size,starts", [((1, 2, 300, 64, 64), [1, 37, 63, 64, 65, 130, 299]), ((2, 2, 700, 128, 128), [200, 448, 500]),
                                         ((1, 1, 9000, 64, 128), [5, 1000, 1001, 4095, 4096, 4097, 6000, 8192]),
                                         ((1, 2, 500, 40, 24), [250, 256, 264, 480])])
def test_gradients_over_documents(size, starts, dtype):
    x = make(*size, dtype, s0=True, seed=31)
    documents(x, starts)
    x[3][0, 0, 20] = -205.0  # acts as -inf
    g = torch.Generator().manual_seed(32)
    dO = torch.randn(x[2].shape, generator=g).to(dtype).cuda()
    dS = 0.3 * torch.randn(x[4].shape, generator=g).cuda()
    check(x, dO, dS, decay.decay_bwd(*x[:4], dO, x[4], dS))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,L", [(64, 400), (128, 9000), (40, 400)])
def test_a_document_without_a_gradient_has_none(d, L, dtype):
    """What is behind a token that forgets does not reach the tokens in front of it, nor does its rounding."""
    x = make(1, 2, L, d, d, dtype, s0=True, seed=33)
    docs = documents(x, [3, 70, 190, L // 2, L - 60])
    g = torch.Generator().manual_seed(34)
    dO = torch.randn(x[2].shape, generator=g).to(dtype).cuda()
    dS = torch.randn(x[4].shape, generator=g).cuda()
    quiet = docs[1::2]
    for a, b in quiet:
        dO[:, :, a:b] = 0
    got = decay.decay_bwd(*x[:4], dO, x[4], dS)
    for a, b in quiet[:-1] if docs[-1] in quiet else quiet:  # dS reaches the last one
        assert not any(bool(t[:, :, a:b].any()) for t in got[:4])


@pytest.mark.parametrize("dtype,size", [(BF, (1, 2, 16384, 128, 128)), (BF, (1, 1, 65536, 128, 64)), (BF, (1, 1, 65536, 64, 64)),
                                        (F32, (1, 1, 20000, 64, 64))])
@pytest.mark.parametrize("level", [1.0, 5.0])
def test_gradients_of_long_rows(size, dtype, level):
    """Heads that remember some 4 and some 150 tokens.  dl's errors do not grow with the row."""
    x = make(*size, dtype, seed=35, level=level)
    dO = torch.randn(x[2].shape, generator=torch.Generator().manual_seed(36)).to(dtype).cuda()
    check(x, dO, None, decay.decay_bwd(*x[:4], dO))


def test_gradients_past_32_bits():
    """More than 2^31 elements a tensor: the last head's end, where nothing behind it and e^-40 in front of it counts,
    is that of a run alone."""
    H, L, d = 17, 1 << 20, 128
    g = torch.Generator(device="cuda").manual_seed(37)
    q, k, v, dO = (torch.empty(1, H, L, d, dtype=BF, device="cuda").normal_(std=0.1, generator=g) for _ in range(4))
    l = torch.full((1, H, L), -0.01, dtype=BF, device="cuda")
    got = decay.decay_bwd(q, k, v, l, dO)
    n, m = 5000, 1000
    tail = [t[:, -1:, -n:].contiguous() for t in (q, k, v, l)]
    ref = walked_gradients(*tail, None, dO[:, -1:, -n:].contiguous(), None)
    for a, b in zip(got[:3], ref[:3]):
        near(a[:, -1:, -m:], b[:, :, -m:], OUT[BF])
    near(got[3][:, -1:, -m:], ref[3][:, :, -m:], DL[BF])
    assert efla.last_device_error() == 0
