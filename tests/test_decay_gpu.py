"""Decayed linear attention on the GPU against the token recurrence in 64 bits.

Tolerances, in half steps u of a type (bf16 2^-8, fp32 2^-24), as a relative 2-norm; a single element may
be off by eight times that of max(rms, |value|):
  fp32 (inputs, states): a value is a sum of up to 64 products per chunk and 128 for the state's share,
  each rounded by at most u, plus the decays (a few u): 64 u covers the sum of their squares' roots
  (sqrt(192) ~ 14 u) with room for the carried state.
  bf16 outputs: the final rounding is at most u of every element; the operands that are rounded on the way
  (the masked products and the state's copy) are off by at most u each, in terms that add like the value
  itself: 2 u together.  States are carried in fp32 from products rounded at 2^-16 (a split in two bf16
  halves) or finer: 2^-16 relative.
"""
import pytest
import torch

import decay_ref as R
from delta_rule_linear_efla_b200 import decay, efla

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
OUT = {BF: 2 * 2.0 ** -8, F32: 64 * 2.0 ** -24}
STATE = {BF: 2.0 ** -16, F32: 64 * 2.0 ** -24}


def near(x, ref, tol):
    rel, big = R.far(x, ref)
    assert rel <= tol and big <= 8 * tol, (rel, big, tol)


def make(B, H, L, dk, dv, dtype, form="token", s0=False, seed=0, level=3.0):
    g = torch.Generator().manual_seed(seed)

    def n(*shape, std=1.0):
        return std * torch.randn(shape, generator=g)

    q, k, v = n(B, H, L, dk, std=dk ** -0.5), n(B, H, L, dk, std=dk ** -0.5), n(B, H, L, dv)
    if form == "head":
        l = torch.log1p(-torch.exp2(-1.0 - 8.0 * torch.rand(H, generator=g))).cuda()
    else:
        l = torch.nn.functional.logsigmoid(level + n(B, H, L)).to(dtype).cuda()
    S0 = n(B, H, dk, dv, std=0.3).cuda() if s0 else None
    return [t.to(dtype).cuda() for t in (q, k, v)] + [l, S0]


SIZES = [(1, 1, 1, 64, 64), (2, 3, 63, 64, 64), (1, 2, 64, 128, 128), (1, 2, 65, 128, 64), (2, 1, 200, 64, 128),
         (1, 3, 130, 40, 24), (1, 2, 333, 17, 33), (1, 1, 70, 1, 1), (1, 1, 1000, 128, 128), (1, 2, 2100, 64, 64),
         (40, 4, 130, 128, 128), (5, 13, 1500, 64, 64), (1, 149, 700, 64, 128)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("form,s0", [("token", False), ("token", True), ("head", True)])
@pytest.mark.parametrize("size", SIZES)
def test_forward(size, form, s0, dtype):
    x = make(*size, dtype, form, s0, seed=sum(size))
    o, S = decay.decay_chunk_fwd(*x)
    ro, rS = R.recurrence(*x)
    assert o.dtype == dtype and S.dtype == F32
    near(o, ro, OUT[dtype])
    near(S, rS, STATE[dtype])
    assert efla.last_device_error() == 0


@pytest.mark.parametrize("size", [(1, 2, 300, 128, 128), (1, 2, 100, 48, 80)])
def test_output_types(size):
    for dtype, o_dtype in ((BF, F32), (F32, BF)):
        x = make(*size, dtype, "token", True)
        o, _ = decay.decay_chunk_fwd(*x, o_dtype=o_dtype)
        assert o.dtype == o_dtype
        near(o, R.recurrence(*x)[0], OUT[BF])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128, 40])
def test_documents_in_a_row(dtype, d):
    """-inf forgets: every document's outputs are those of a run of its own, and what lies below -200 acts alike."""
    x = make(1, 2, 400, d, d, dtype, s0=True, seed=5)
    cuts = [0, 1, 2, 63, 64, 65, 190, 191, 399]
    x[3][:, :, cuts] = float("-inf")
    x[3][:, :, 300] = -250.0
    o, S = decay.decay_chunk_fwd(*x)
    ro, rS = R.recurrence(*x)
    near(o, ro, OUT[dtype])
    near(S, rS, STATE[dtype])
    a, b = 65, 190
    alone, _ = decay.decay_chunk_fwd(*(t[:, :, a:b].contiguous() for t in x[:4]))
    near(o[:, :, a:b], alone.double(), 2 * OUT[dtype])
    x[3][:] = float("-inf")  # nothing but the token itself
    o, S = decay.decay_chunk_fwd(*x)
    near(o, (x[0].double() * x[1].double()).sum(-1, keepdim=True) * x[2].double(), OUT[dtype])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strong_and_weak_decays_mixed(dtype):
    """Weak decays behind strong ones in the same chunk keep their precision (sums of logs in the thousands)."""
    x = make(1, 2, 256, 64, 64, dtype, seed=6, level=6.0)
    x[3][:, :, ::16] = -150.0
    o, S = decay.decay_chunk_fwd(*x)
    ro, rS = R.recurrence(*x)
    near(o, ro, OUT[dtype])
    near(S, rS, STATE[dtype])


def test_no_decay_and_growth():
    x = make(1, 2, 200, 64, 64, F32, seed=7)
    x[3][:] = 0.0
    near(decay.decay_chunk_fwd(*x)[0], R.recurrence(*x)[0], OUT[F32])
    x[3][:] = 0.01
    near(decay.decay_chunk_fwd(*x)[0], R.recurrence(*x)[0], OUT[F32])


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 24)])
def test_no_tokens_and_in_place_state(dtype, d):
    x = make(1, 2, 0, d, d, dtype, s0=True)
    o, S = decay.decay_chunk_fwd(*x)
    assert o.shape == (1, 2, 0, d) and torch.equal(S, x[4])
    assert not decay.decay_chunk_fwd(*x[:4])[1].any()
    x = make(1, 2, 150, d, d, dtype, s0=True)
    ro, rS = decay.decay_chunk_fwd(*x)
    o, S = decay.decay_chunk_fwd(*x[:4], S0=x[4], S_final=x[4])
    assert S is x[4] and torch.equal(o, ro) and torch.equal(S, rS)
    o, S = decay.decay_chunk_fwd(*x, want_state=False)
    assert S is None


@pytest.mark.parametrize("dtype,size", [(BF, (1, 1, 9000, 64, 128)), (BF, (2, 3, 2000, 128, 128)), (F32, (1, 1, 9000, 16, 24)),
                                        (F32, (1, 2, 3000, 128, 100))])
def test_in_place_state_of_sequences_that_are_cut(dtype, size):
    """Every stretch of a cut sequence starts from S0, whichever of them ends first.  The state remembers up to 141
    chunks: 141 * 2.4e-7 of truncation above the 3e-6 of one, below 4 * 2^-16; in fp32, 141 more roundings of u."""
    q, k, v, l, S0 = make(*size, dtype, s0=True, seed=8)
    l = l / 4096  # S0 counts up to the end
    o, S = decay.decay_chunk_fwd(q, k, v, l, S0)
    near(S, R.recurrence(q, k, v, l, S0)[1], 4 * STATE[dtype])
    for _ in range(20):
        carried = S0.clone()
        o2, S2 = decay.decay_chunk_fwd(q, k, v, l, carried, S_final=carried)
        assert S2 is carried and torch.equal(o, o2) and torch.equal(S, carried)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
def test_prompt_in_two_parts_then_decode(dtype, d):
    """A prompt in two calls, then tokens one at a time, is one call over all of it."""
    x = make(2, 2, 300, d, d, dtype, s0=True, seed=8)
    ro, rS = R.recurrence(*x)
    parts, S = [], x[4]
    for a, b in ((0, 100), (100, 280)):
        o, S = decay.decay_chunk_fwd(*(t[:, :, a:b].contiguous() for t in x[:4]), S)
        parts.append(o)
    for t in range(280, 300):
        o = decay.decay_recurrent_step(*(z[:, :, t].contiguous() for z in x[:4]), S)
        parts.append(o[:, :, None])
    near(torch.cat(parts, 2), ro, OUT[dtype])
    near(S, rS, STATE[dtype])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", [(1, 1, 64, 64), (3, 5, 128, 128), (2, 2, 128, 64), (1, 3, 256, 256), (2, 2, 7, 5),
                                  (1, 2, 33, 250), (1, 1, 1, 1), (70, 16, 128, 128)])
@pytest.mark.parametrize("form", ["token", "head"])
def test_step(size, form, dtype):
    B, H, dk, dv = size
    q, k, v, l, S = make(B, H, 1, dk, dv, dtype, form, True, seed=9)
    if form == "token":
        l[0, 0] = float("-inf")
        l = l[:, :, 0].contiguous()
    args = [t[:, :, 0].contiguous() for t in (q, k, v)]
    ro, rS = R.recurrence(q, k, v, l if form == "head" else l[..., None], S)
    o = decay.decay_recurrent_step(*args, l, S)
    # one product and one sum an element, then a sum over dk <= 256 of them
    near(S, rS, 4 * 2.0 ** -24)
    near(o, ro[:, :, 0], 2.0 ** -8 if dtype == BF else OUT[F32])


GRAD_SIZES = [(1, 1, 1, 64, 64), (1, 2, 65, 64, 64), (1, 2, 200, 128, 128), (1, 1, 130, 128, 64), (2, 1, 100, 64, 128),
              (1, 2, 90, 20, 12), (1, 1, 333, 33, 17), (1, 1, 1100, 64, 64), (24, 8, 70, 128, 128), (5, 13, 1500, 64, 64),
              (3, 25, 900, 64, 128)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("form,s", [("token", True), ("token", False), ("head", True)])
@pytest.mark.parametrize("size", GRAD_SIZES)
def test_gradients(size, form, s, dtype):
    """Every gradient against autograd through the recurrence.  dlog_g is a sum over the tokens behind it
    of differences that cancel; 4x the tolerance of the terms."""
    x = make(*size, dtype, form, s, seed=3 + sum(size))
    if form == "token" and size[2] > 40:
        x[3][0, 0, 37] = float("-inf")
    g = torch.Generator().manual_seed(4)
    dO = torch.randn(x[2].shape, generator=g).to(dtype).cuda()
    dS = 0.3 * torch.randn((size[0], size[1], size[3], size[4]), generator=g).cuda() if s else None
    got = decay.decay_bwd(*x[:4], dO, x[4], dS)
    ref = R.gradients(*x, dO, dS)
    for n, a, b in zip(("dq", "dk", "dv"), got, ref):
        assert a.dtype == dtype, n
        near(a, b, OUT[dtype])
    if form == "head":
        assert got[3] is None
    else:
        ok = torch.isfinite(x[3])
        near(torch.where(ok, got[3].double(), 0.0), torch.where(ok, ref[3], 0.0), 4 * OUT[dtype])
        assert not got[3][~ok].any()
    near(got[4], ref[4], STATE[dtype])
    assert decay.decay_bwd(*x[:4], dO, x[4], dS, want_dS0=False)[4] is None
    assert efla.last_device_error() == 0


def test_gradients_against_differences():
    """Directional differences of the forward itself, float32: (f(x + h d) - f(x - h d)) / 2h = <grad, d>, whose
    rounding is about u |f| sqrt(n) / h ~ 1e-3 of it at h = 1e-2; truncation h^2."""
    x = make(1, 2, 90, 16, 24, F32, s0=True, seed=11)
    g = torch.Generator().manual_seed(5)
    dO, dS = torch.randn(x[2].shape, generator=g).cuda(), torch.randn(x[4].shape, generator=g).cuda()
    grads = decay.decay_bwd(*x[:4], dO, x[4], dS)

    def f(y):
        o, S = decay.decay_chunk_fwd(*y)
        return float((o.double() * dO).sum() + (S.double() * dS).sum())

    for i in range(5):
        d = torch.randn(x[i].shape, generator=g).cuda()
        d = d * (0.1 if i == 3 else 1.0)
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + 1e-2 * d, x[i] - 1e-2 * d
        want = float((grads[i].double() * d).sum())
        size = float((grads[i].double().norm() * d.double().norm()))
        assert abs((f(up) - f(down)) / 2e-2 - want) <= 2e-3 * size


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 16)])
def test_autograd_call(dtype, d):
    x = make(1, 2, 100, d, d, dtype, s0=True, seed=12)
    leaves = [t.requires_grad_(True) for t in x]
    g = torch.Generator().manual_seed(6)
    w = torch.randn(x[2].shape, generator=g).to(dtype).cuda()
    o, S = decay.decay_attention(*leaves)
    (o * w).sum().backward()  # S unused: no gradient comes from it
    ref = decay.decay_bwd(*(t.detach() for t in x[:4]), w, x[4].detach())
    for a, b in zip(leaves, ref):
        assert torch.equal(a.grad, b)
    for t in leaves:
        t.grad = None
    _, S = decay.decay_attention(*leaves)
    S.sum().backward()  # the state alone
    assert not leaves[0].grad.any() and torch.isfinite(leaves[1].grad).all() and leaves[1].grad.any()


def test_no_tokens_backward():
    x = make(1, 2, 0, 64, 64, BF, s0=True)
    dS = torch.randn_like(x[4])
    got = decay.decay_bwd(*x[:4], x[2], x[4], dS)
    assert torch.equal(got[4], dS) and got[0].numel() == 0
    assert not decay.decay_bwd(*x[:4], x[2], x[4], None)[4].any()


def _capture(fn):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fn()
    return graph, out


@pytest.mark.parametrize("dtype,size", [(BF, (1, 2, 1500, 128, 128)), (BF, (1, 2, 300, 64, 128)), (F32, (1, 2, 700, 32, 48))])
def test_captured_and_replayed(dtype, size):
    """Two captured graphs, replayed in turn and again, give the eager call's bits."""
    a, b = make(*size, dtype, s0=True, seed=13), make(*size, dtype, s0=True, seed=14)
    dO = torch.randn(a[2].shape, device="cuda").to(dtype)

    def run(x):
        return (*decay.decay_chunk_fwd(*x), *decay.decay_bwd(*x[:4], dO, x[4], x[4]))

    ra, rb = run(a), run(b)
    ga, oa = _capture(lambda: run(a))
    gb, ob = _capture(lambda: run(b))
    for _ in range(2):
        ga.replay()
        gb.replay()
    torch.cuda.synchronize()
    for got, ref in ((oa, ra), (ob, rb)):
        for x, y in zip(got, ref):
            assert torch.equal(x, y)


def test_two_streams_at_once():
    xs = [make(1, 2, 1200, 128, 128, BF, seed=20 + i) for i in range(2)]
    refs = [decay.decay_chunk_fwd(*x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [decay.decay_chunk_fwd(*x, stream=s) for _ in range(3) for x, s in zip(xs, streams)][-2:]
    torch.cuda.synchronize()
    for a, b in zip(got, refs):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("d", [64, 128, 33])
def test_pointers_aligned_to_their_element(d):
    """Dense tensors that start on an odd element."""
    x = make(1, 2, 150, d, d, BF, seed=15)

    def odd(t):
        s = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        s[1:].copy_(t.reshape(-1))
        return s[1:].view(t.shape)

    y = [odd(t) for t in x[:4]]
    near(decay.decay_chunk_fwd(*y)[0], R.recurrence(*x)[0], OUT[BF])
    dO = torch.randn_like(x[2])
    for a, b in zip(decay.decay_bwd(*y, odd(dO)), R.gradients(*x, dO, None)):
        near(a, b, 4 * OUT[BF])


def test_offsets_past_32_bits():
    """More than 2^31 elements a tensor: the last head, and a long sequence's end, are those of a run alone."""
    H, L, d = 17, 1 << 20, 128
    q, k, v = (torch.empty(1, H, L, d, dtype=BF, device="cuda").normal_(std=0.1) for _ in range(3))
    l = torch.full((1, H, L), -0.01, dtype=BF, device="cuda")
    o, S = decay.decay_chunk_fwd(q, k, v, l)
    n = 4000  # e^-40 of what came before
    tail = [t[:, -1:, -n:].contiguous() for t in (q, k, v, l)]
    ro, rS = R.recurrence(*tail)
    near(o[:, -1:, -500:], ro[:, :, -500:], OUT[BF])
    near(S[:, -1:], rS, STATE[BF])


@pytest.mark.parametrize("size", [(3, 25, 900, 64, 128), (3, 25, 900, 128, 64), (4, 16, 1000, 128, 128), (1, 149, 700, 64, 128)])
def test_repeats_give_the_same_bits_without_a_wait_that_gave_up(size):
    """Cut sequences, several walks to a CTA: forty repeats of forward and backward, bit for bit."""
    x = make(*size, BF, seed=17)
    dO = torch.randn(x[2].shape, device="cuda").to(BF)

    def run():
        return [t for t in (*decay.decay_chunk_fwd(*x), *decay.decay_bwd(*x[:4], dO)) if t is not None]

    ref = run()
    for _ in range(40):
        for a, b in zip(run(), ref):
            assert torch.equal(a, b)
    assert efla.last_device_error() == 0


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 32)])
def test_a_log_decay_that_is_not_a_number_reaches_later_tokens_only(dtype, d):
    x = make(1, 2, 1500, d, d, dtype, s0=True, seed=18)
    ref, _ = decay.decay_chunk_fwd(*x)
    at = 700
    x[3][0, 1, at] = float("nan")
    o, S = decay.decay_chunk_fwd(*x)
    assert torch.equal(o[0, 0], ref[0, 0]) and torch.equal(o[0, 1, :at], ref[0, 1, :at])
    assert torch.isnan(o[0, 1, at:]).all() and torch.isnan(S[0, 1]).all() and torch.isfinite(S[0, 0]).all()


def test_rows_behind_the_output_are_left_alone():
    x = make(1, 1, 70, 128, 128, BF, seed=16)
    buf = torch.full((2 * 70 * 128,), 7.0, dtype=BF, device="cuda")
    o, _ = decay.decay_chunk_fwd(*x, o=buf[: 70 * 128].view(1, 1, 70, 128))
    near(o, R.recurrence(*x)[0], OUT[BF])
    assert (buf[70 * 128 :] == 7).all()
