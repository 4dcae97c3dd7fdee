"""Layer norm against its fp64 statement.  Bounds per element: half a step of
the output's type, and for the fp32 arithmetic 2^-18 of the terms' magnitudes
(a sum of up to 2^14 features runs through at most 16 serial and 10 tree
additions, 2^-24 each, with the few products before and after it)."""
import numpy as np
import pytest

from oracle import attn_block_oracle as O
from tests import gpu_cases as G

pytestmark = pytest.mark.gpu

HALF, FP = 2.0 ** -8, 2.0 ** -18


def _inputs(M, d, seed, f32, offset=0.5):
    import torch
    gen = torch.Generator().manual_seed(seed)
    scale = 2.0 ** torch.randint(-6, 7, (M, 1), generator=gen)
    X = ((torch.randn(M, d, generator=gen) + offset * torch.randn(M, 1, generator=gen)) * scale).bfloat16()
    g = (0.5 + torch.rand(d, generator=gen)).bfloat16()
    b = torch.randn(d, generator=gen).bfloat16()
    dY = torch.randn(M, d, generator=gen)
    return X, g, b, dY if f32 else dY.bfloat16()


def _close(name, got, want, bound):
    off = np.abs(G.host_f64(got) - want)
    worst = (off / bound).max() if off.size else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} times its bound"


SHAPES = [(1, 8), (1, 4096), (3, 72), (37, 264), (9, 512), (9, 520), (65, 1024), (33, 1032), (5, 2056), (130, 4096),
          (7, 4104), (600, 5120), (3, 8200), (40, 14336), (5, 16384)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,d", SHAPES)
def test_layer_norm(M, d, f32):
    import lora_linear_fine_b200 as L
    X, g, b, dY = _inputs(M, d, 11 * d + M, f32)
    eps = 1e-5
    shift = None if f32 else b
    Y, mean, rstd = L.layer_norm(X.cuda(), g.cuda(), None if shift is None else b.cuda(), eps)
    dX, dg, db = L.layer_norm_backward(dY.cuda(), X.cuda(), g.cuda(), mean, rstd, bias=not f32)
    x, gg, dy = G.host_f64(X), G.host_f64(g), G.host_f64(dY)
    bb = None if shift is None else G.host_f64(b)
    e32 = float(np.float32(eps))
    y_ref, mean_ref, rstd_ref = O.layer_norm(x, gg, bb, e32)
    xh = (x - mean_ref[:, None]) * rstd_ref[:, None]
    # |x| rstd: what the mean's own error and the subtraction scale with
    size = (np.abs(x) + np.abs(x).mean(1)[:, None]) * rstd_ref[:, None]
    _close("mean", mean, mean_ref, FP * np.abs(x).mean(1) + 1e-30)
    # var is off by its own arithmetic and by (the mean's error)^2; relative
    _close("rstd", rstd, rstd_ref, rstd_ref * (FP + (FP * size.mean(1)) ** 2))
    _close("Y", Y, y_ref, HALF * np.abs(y_ref) + FP * (size * np.abs(gg) + (0 if bb is None else np.abs(bb))) + 1e-38)
    dX_ref, dg_ref, db_ref = O.layer_norm_backward(dy, x, gg, e32)
    dh = np.abs(dy * gg)
    xs = np.abs(xh) + FP * size
    terms = rstd_ref[:, None] * (dh + dh.mean(1)[:, None] + xs * (dh * xs).mean(1)[:, None] +
                                 size * (dh * xs).mean(1)[:, None] + xs * (dh * size).mean(1)[:, None])
    _close("dX", dX, dX_ref, HALF * np.abs(dX_ref) + FP * terms + 1e-38)
    # a column's sum adds at most M rows one after the other
    sums = M * 2.0 ** -24 + FP
    _close("dg", dg, dg_ref, sums * (np.abs(dy) * (np.abs(xh) + size)).sum(0) + 1e-38)
    if f32:
        assert db is None
    else:
        _close("db", db, db_ref, sums * np.abs(dy).sum(0) + 1e-38)


def test_constant_rows_and_no_eps():
    """A row of one value has variance 0: y is the shift, and with eps its gradient stays finite."""
    import lora_linear_fine_b200 as L
    import torch
    X = torch.full((2, 264), 3.0, dtype=torch.bfloat16, device="cuda")
    g, b = torch.ones(264, dtype=torch.bfloat16, device="cuda"), torch.full((264,), 0.25, dtype=torch.bfloat16, device="cuda")
    Y, mean, rstd = L.layer_norm(X, g, b, 1e-5)
    assert torch.all(Y == 0.25) and torch.all(mean == 3.0)
    dX, _, _ = L.layer_norm_backward(torch.randn(2, 264, device="cuda").bfloat16(), X, g, mean, rstd)
    assert torch.isfinite(dX).all()


def test_no_tokens():
    import lora_linear_fine_b200 as L
    import torch
    X, g = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, dtype=torch.bfloat16, device="cuda")
    Y, mean, rstd = L.layer_norm(X, g)
    dX, dg, db = L.layer_norm_backward(X, X, g, mean, rstd)
    assert Y.shape == dX.shape == (0, 64) and not dg.any() and not db.any()


def test_in_place_and_partial_gradients():
    """Y may be X; dX may be dY; dg or db alone."""
    import lora_linear_fine_b200 as L
    import torch
    X, g, b, dY = (t.cuda() for t in _inputs(300, 4096, 5, False))
    Y, mean, rstd = L.layer_norm(X, g, b)
    dX, dg, db = L.layer_norm_backward(dY, X, g, mean, rstd)
    st = torch.cuda.current_stream().cuda_stream
    ws = L.Workspace(L.lora_linear_layernorm_workspace_size(300, 4096))
    for want in ((True, False), (False, True), (False, False)):
        g2, b2 = torch.full_like(dg, 7.0), torch.full_like(db, 7.0)
        d2 = dY.clone()
        assert L.lora_linear_layernorm_bwd(d2.data_ptr(), 0, X.data_ptr(), g.data_ptr(), mean.data_ptr(),
                                           rstd.data_ptr(), 300, 4096, d2.data_ptr(),
                                           g2.data_ptr() if want[0] else None, b2.data_ptr() if want[1] else None,
                                           ws.buf.data_ptr(), ws.nbytes, st) == 0
        assert torch.equal(d2, dX)
        assert torch.equal(g2, dg if want[0] else torch.full_like(dg, 7.0))
        assert torch.equal(b2, db if want[1] else torch.full_like(db, 7.0))
    x2 = X.clone()
    assert L.lora_linear_layernorm_fwd(x2.data_ptr(), g.data_ptr(), b.data_ptr(), 300, 4096, 1e-5, x2.data_ptr(),
                                       mean.data_ptr(), rstd.data_ptr(), st) == 0
    assert torch.equal(x2, Y)


def test_same_bits_graph_and_stream():
    """Every call gives the same bits: again, captured and replayed on new inputs, and on another stream."""
    import lora_linear_fine_b200 as L
    import torch
    X, g, b, dY = (t.cuda() for t in _inputs(1000, 1032, 6, False))
    ws = L.Workspace(L.lora_linear_layernorm_workspace_size(1000, 1032))

    def step(stream=None):
        Y, mean, rstd = L.layer_norm(X, g, b, stream=stream)
        return (Y, mean, rstd) + L.layer_norm_backward(dY, X, g, mean, rstd, workspace=ws, stream=stream)

    first = step()
    assert all(torch.equal(p, q) for p, q in zip(first, step()))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = step(side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    X.mul_(-2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(held, step()))


def test_offsets_past_32_bits():
    """The last rows of a matrix of more than 2^31 elements."""
    import lora_linear_fine_b200 as L
    import torch
    M, d = (1 << 31) // 8192 + 300, 8192
    X = torch.zeros(M, d, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(5, d, device="cuda").bfloat16()
    X[-5:] = tail
    g = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    Y, mean, rstd = L.layer_norm(X, g)
    y, m, r = L.layer_norm(tail, g)
    assert torch.equal(Y[-5:], y) and torch.equal(mean[-5:], m) and torch.equal(rstd[-5:], r)
    dX, dg, _ = L.layer_norm_backward(X, X, g, mean, rstd)
    dx, dg2, _ = L.layer_norm_backward(tail, tail, g, m, r)
    assert torch.equal(dX[-5:], dx) and torch.allclose(dg, dg2, rtol=1e-5, atol=1e-5)
