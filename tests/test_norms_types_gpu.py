"""The norms where a result has more bits than the gate."""
import pytest
import torch

import decay_ref as R
from delta_rule_linear_efla_b200 import norms

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_fp32_gradient_under_bf16_gates_far_below_zero(act):
    """d_o is float32 where o is, whatever the gate's type.  One element of each row carries a gradient, so that its
    d_o = r dn (1 - n^2 / d) cancels little: in half steps u = 2^-24, the sigmoid is off by 6 (an exponential within 2
    ulp, a sum, a division), dn by 10, r by 12 (a sum of 64 squares in turns and pairs, halved by the root, which is
    within 2 ulp), the product by 1, and the correction of at most an eighth by 64 of its own: below 32 u."""
    gates = torch.arange(-85, -2, 0.25).to(torch.bfloat16).cuda()
    n, d = gates.numel(), 64
    g = torch.Generator().manual_seed(1)
    o = (0.5 + torch.rand((1, 1, n, d), generator=g)).cuda()
    gate = gates[None, :, None, None].expand(1, n, 1, d).contiguous()
    dy = torch.zeros_like(gate)
    dy[..., 5] = 1.0
    got = norms.gated_norm_bwd(o, gate, dy, act=act)[0]
    leaf = o.double().requires_grad_(True)
    ref = torch.autograd.grad(R.gated_norm(leaf, gate, None, None, 1.0, 1e-6, act), leaf, dy.double())[0]
    assert got.dtype is torch.float32
    off = float(((got.double() - ref) / ref).abs()[..., 5].max())
    assert off <= 32 * 2.0 ** -24
