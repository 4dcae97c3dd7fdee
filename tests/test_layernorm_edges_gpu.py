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


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("value", [1000.0, 29952.0, 0.1])
@pytest.mark.parametrize("d", DIMS)
def test_gradients_of_constant_rows(d, value, f32):
    """x_hat is zero, so dg is, and dX is rstd (dh - mean(dh)): half a step of
    bf16 and 2^-18 of the terms, as in the other tests of the layer norm."""
    import lora_linear_fine_b200 as L
    X, g, b, dY = _constant(d, value)
    dY = dY.float() if f32 else dY
    _, mean, rstd = L.layer_norm(X, g, b, 1e-5)
    dX, dg, db = L.layer_norm_backward(dY, X, g, mean, rstd)
    assert not dg.any()
    dh = G.host_f64(dY) * G.host_f64(g)
    rs = 1e-5 ** -0.5
    want = rs * (dh - dh.mean(1)[:, None])
    bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * rs * (np.abs(dh) + np.abs(dh).mean(1)[:, None])
    assert (np.abs(G.host_f64(dX) - want) <= bound).all()


@pytest.mark.parametrize("d", [1000, 4096])
def test_rows_far_from_zero(d):
    """Rows of two values one step of bf16 apart around 2^10: x - mean is exact
    here (both are multiples of 2^-12 below 2^12), so x_hat keeps all its bits:
    dg of one row is dY x_hat to a handful of half steps of 2^-24."""
    import lora_linear_fine_b200 as L
    import torch
    gen = torch.Generator().manual_seed(d)
    X = 1024.0 + 8.0 * (torch.arange(d) % 2).float()[None, :]
    X = X.bfloat16().cuda()
    g = (0.5 + torch.rand(d, generator=gen)).bfloat16().cuda()
    dY = torch.randn(1, d, generator=gen).bfloat16().cuda()
    _, mean, rstd = L.layer_norm(X, g, None, 1e-5)
    assert float(mean) == 1028.0
    _, dg, _ = L.layer_norm_backward(dY, X, g, mean, rstd)
    xh = (G.host_f64(X) - 1028.0) / (16.0 + float(np.float32(1e-5))) ** 0.5
    want = (G.host_f64(dY) * xh)[0]
    assert (np.abs(G.host_f64(dg) - want) <= 2.0 ** -21 * np.abs(want)).all()
