"""Layer norm of rows whose values are all the same, or nearly so."""
import numpy as np
import pytest

from tests import gpu_cases as G

pytestmark = pytest.mark.gpu

DIMS = [264, 1000, 1032, 4096, 5120, 14336]


def _constant(d, value):
    import torch
    gen = torch.Generator().manual_seed(d)
    X = torch.full((5, d), value, dtype=torch.bfloat16)
    X[3] *= -0.25
    g = (0.5 + torch.rand(d, generator=gen)).bfloat16()
    b = torch.randn(d, generator=gen).bfloat16()
    return X.cuda(), g.cuda(), b.cuda(), torch.randn(5, d, generator=gen).bfloat16().cuda()


@pytest.mark.parametrize("value", [1000.0, 29952.0, 0.1, -7.0])
@pytest.mark.parametrize("d", DIMS)
def test_constant_rows(d, value):
    """A row of one value: its sum is exact in fp32 (d times 8 bits), so its
    mean is the value and Y the shift, exactly."""
    import lora_linear_fine_b200 as L
    import torch
    X, g, b, _ = _constant(d, value)
    Y, mean, rstd = L.layer_norm(X, g, b, 1e-5)
    assert torch.equal(mean, X[:, 0].float())
    assert torch.equal(Y, b.expand(5, d))
    assert np.abs(G.host_f64(rstd) * 1e-5 ** 0.5 - 1).max() <= 2.0 ** -20
