"""The reference for long rows against autograd, on the CPU."""
import torch

import decay_ref as R
from decay_walked_ref import walked_gradients


def test_walked_reference_gradients():
    """The reference for long rows is autograd's through the recurrence, over several documents too."""
    g = torch.Generator().manual_seed(2)

    def n(*s):
        return torch.randn(s, generator=g, dtype=torch.float64)

    x = [n(1, 2, 9, 3), n(1, 2, 9, 3), n(1, 2, 9, 4), -n(1, 2, 9).abs(), n(1, 2, 3, 4)]
    x[3][0, 0, 4] = x[3][0, 1, 2] = x[3][0, 1, 7] = -300.0
    dO, dS = n(1, 2, 9, 4), n(1, 2, 3, 4)
    for args in ((x[4], dO, dS), (None, dO, None)):
        for a, b in zip(walked_gradients(*x[:4], *args), R.gradients(*x[:4], *args)):
            assert (a - b).abs().max() <= 1e-12
