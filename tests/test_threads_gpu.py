"""Calls from host threads at once: what one sets up for its launch does not reach the other's."""
import threading

import pytest
import torch

from delta_rule_linear_efla_b200 import decay, efla

pytestmark = pytest.mark.gpu


def _decay(d, g):
    """(call, its output) of the forward with prepared arguments, straight into the library: little else is done
    between two calls, so that threads meet within them."""
    q, k, v = ((0.2 * torch.randn((1, 2, 130, d), generator=g)).cuda() for _ in range(3))
    l = torch.nn.functional.logsigmoid(3 + torch.randn((1, 2, 130), generator=g)).cuda()
    need = decay.decay_workspace_size(1, 2, 130, d, d, q.dtype)
    ws, o = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda"), torch.empty_like(v)
    p, f = [t.data_ptr() for t in (q, k, v, l)], efla.load_library().efla_decay_chunk_fwd

    def call(stream):
        return f(*p, 0, None, o.data_ptr(), None, 1, 2, 130, d, d, efla.EFLA_F32, efla.EFLA_F32, ws.data_ptr(), need, stream)

    call.keep = (q, k, v, l, ws)
    return call, o


def _delta(d, g):
    q, k, v = ((0.2 * torch.randn((1, 2, 130, d), generator=g)).cuda() for _ in range(3))
    beta, o = torch.rand((1, 2, 130), generator=g).cuda(), torch.empty_like(v)
    p, f = [t.data_ptr() for t in (q, k, v, beta)], efla.load_library().efla_chunk_fwd

    def call(stream):
        return f(*p, None, o.data_ptr(), None, 1, 2, 130, d, d, 64, efla.EFLA_F32, efla.EFLA_F32, None, 0, stream)

    call.keep = (q, k, v, beta)
    return call, o


@pytest.mark.parametrize("make", [_decay, _delta])
def test_host_threads_with_other_head_sizes(make):
    """Head sizes 128 and 16 in fp32 share their kernels, and need other amounts of shared memory."""
    g = torch.Generator().manual_seed(1)
    calls = [make(d, g) for d in (128, 16, 128, 16)]
    refs = []
    for c, o in calls:
        assert c(None) == 0
        torch.cuda.synchronize()
        refs.append(o.clone())
    streams = [torch.cuda.Stream() for _ in calls]
    start, refused = threading.Barrier(len(calls)), []

    def work(call, stream):
        start.wait()
        refused.append(sum(call(stream) != 0 for _ in range(10000)))

    threads = [threading.Thread(target=work, args=(c, s.cuda_stream)) for (c, _), s in zip(calls, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert refused == [0] * len(calls)
    assert all(torch.equal(o, r) for (_, o), r in zip(calls, refs))
