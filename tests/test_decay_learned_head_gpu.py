"""A learned log-decay for each head, given for every token as the refusal of a [H] one says."""
import re

import pytest
import torch

import decay_ref as R
from delta_rule_linear_efla_b200 import decay
from test_decay_gpu import BF, F32, OUT, make, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
def test_what_the_refusal_says_works(dtype):
    q, k, v, log_g, _ = make(2, 3, 130, 64, 64, dtype, "head", seed=41)
    log_g.requires_grad_(True)
    with pytest.raises(ValueError, match="no gradient") as e:
        decay.decay_attention(q, k, v, log_g)
    says = re.search(r"log_g\[.*", str(e.value)).group(0)
    B, H, L, _ = q.shape
    given = eval(says, dict(log_g=log_g, q=q, B=B, H=H, L=L))
    dO = torch.randn(v.shape, generator=torch.Generator().manual_seed(42)).to(dtype).cuda()
    o, _ = decay.decay_attention(q, k, v, given)
    (o * dO).sum().backward()
    ref = R.gradients(q, k, v, given.detach(), None, dO, None)[3].sum((0, 2))
    # a sum over 260 tokens of gradients within their tolerance, and its own rounding to the type on the way back
    near(log_g.grad, ref, 4 * OUT[dtype])
