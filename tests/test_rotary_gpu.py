"""Rotary tables and the rotation of finished q and k against their fp64
statements.  Bounds per element: half a step of the output's type, and 2^-22
of the terms for the fp32 products and the sum (three roundings of 2^-24); the
tables are within 2^-22 of their amplitude (the remainder of a turn is rounded
once to fp32, a relative 2^-24 of at most pi, and the sine and cosine of it
are good to a few units in the last place)."""
import numpy as np
import pytest

from oracle import attn_block_oracle as O
from tests import gpu_cases as G

pytestmark = pytest.mark.gpu

SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0, base=500000.0),
            dict(scaling="wavelength", factor=8.0, low=1.0, high=4.0, original=8192, base=500000.0),
            dict(scaling="ramp", factor=16.0, low=1.0, high=32.0, original=4096, amplitude=1.2772588722239782)]


@pytest.mark.parametrize("kw", SCALINGS, ids=lambda k: k.get("scaling", "none"))
@pytest.mark.parametrize("n_pos,rot", [(1, 16), (1000, 48), (4097, 128), (200, 256)])
def test_tables(n_pos, rot, kw):
    import lora_linear_fine_b200 as L
    cos, sin = L.rotary_tables(n_pos, rot, **kw)
    c, s = O.rotary_tables(n_pos, rot, **kw)
    bound = 2.0 ** -21 * kw.get("amplitude", 1.0)
    assert np.abs(G.host_f64(cos) - c).max() <= bound and np.abs(G.host_f64(sin) - s).max() <= bound


def test_tables_far_positions():
    """Position 2^20 - 1 of the fastest pair: an angle of 10^6 rad."""
    import lora_linear_fine_b200 as L
    n = 1 << 20
    cos, sin = L.rotary_tables(n, 16, scaling="wavelength", factor=2.0, original=65536)
    f = O.rotary_frequencies(16, scaling="wavelength", factor=2.0, original=65536)
    at = np.arange(n - 1000, n, dtype=np.float64)[:, None] * f
    assert np.abs(G.host_f64(cos[-1000:]) - np.cos(at)).max() <= 2.0 ** -21
    assert np.abs(G.host_f64(sin[-1000:]) - np.sin(at)).max() <= 2.0 ** -21


def _case(M, heads, kv, hd, rot, n_pos, seed):
    import torch
    gen = torch.Generator().manual_seed(seed)
    Q = torch.randn(M, heads * hd, generator=gen).bfloat16().cuda()
    K = torch.randn(M, kv * hd, generator=gen).bfloat16().cuda() if kv else None
    pos = torch.randint(0, n_pos, (M,), generator=gen, dtype=torch.int32).cuda()
    return Q, K, pos


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("M,heads,kv,hd,rot", [(1, 1, 1, 16, 16), (1, 32, 8, 128, 128), (37, 5, 0, 80, 32), (3, 9, 3, 24, 16),
                                               (200, 7, 2, 256, 256), (129, 4, 4, 64, 48), (1000, 16, 16, 96, 96)])
def test_rotary(M, heads, kv, hd, rot, layout, inverse):
    import lora_linear_fine_b200 as L
    import torch
    Q, K, pos = _case(M, heads, kv, hd, rot, 300, M + hd)
    cos, sin = L.rotary_tables(300, rot, amplitude=1.1)
    ws = L.Workspace(256)
    Yq, Yk = L.rotary(Q, K, pos, cos, sin, hd, layout, inverse, workspace=ws)
    p, c, s = pos.cpu().numpy(), G.host_f64(cos), G.host_f64(sin)
    for x, y in ((Q, Yq), (K, Yk)):
        if x is None:
            assert y is None
            continue
        ref = O.rotary(G.host_f64(x), p, c, s, hd, layout, inverse)
        size = O.rotary(np.abs(G.host_f64(x)), p, np.abs(c), -np.abs(s), hd, layout) + \
            O.rotary(np.abs(G.host_f64(x)), p, np.abs(c), np.abs(s), hd, layout)
        off = np.abs(G.host_f64(y) - ref)
        assert (off <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -21 * np.abs(size) + 1e-38).all()
        kept = np.arange(heads * hd if x is Q else kv * hd) % hd >= rot
        assert torch.equal(x.cpu()[:, kept], y.cpu()[:, kept])
    qi, ki = Q.clone(), None if K is None else K.clone()
    L.rotary(qi, ki, pos, cos, sin, hd, layout, inverse, inplace=True, workspace=ws)
    assert torch.equal(qi, Yq) and (K is None or torch.equal(ki, Yk))
    assert ws.status() == 0


def test_agrees_with_the_fused_rotation():
    """A projection's rotary epilogue and the rotation of the finished
    projection differ by the rounding in between: half a step of each of the
    pair, turned, and half a step of both results."""
    import lora_linear_fine_b200 as L
    import seeded_inputs as S
    import torch
    M, d, hd = 100, 256, 64
    t = {k: G.dev(v) for k, v in S.make_inputs(M, d, 256, 8, "identity", seed=3).items()}
    cos, sin = L.rotary_tables(64, hd)
    pos = torch.from_numpy(S.draw_positions(M, 64, 3)).cuda()
    desc = L.make_desc(M, d, 256, 8, 2.0, "identity")
    ws = L.Workspace(L.lora_linear_workspace_size_rope(desc, 0))
    Y = torch.empty(M, 256, dtype=torch.bfloat16, device="cuda")
    rope = L.make_rope_desc(pos.data_ptr(), cos.data_ptr(), sin.data_ptr(), 64, hd)
    assert L.lora_linear_fwd_rope(desc, rope, t["X"].data_ptr(), t["W"].data_ptr(), t["A"].data_ptr(),
                                  t["B"].data_ptr(), Y.data_ptr(), None, ws.buf.data_ptr(), ws.nbytes,
                                  torch.cuda.current_stream().cuda_stream) == 0
    Z, _, _ = L.forward(t["X"], t["W"], t["A"], t["B"], 2.0)
    R, _ = L.rotary(Z, None, pos, cos, sin, hd)
    z = np.abs(G.host_f64(Z)).reshape(M, -1, 2, hd // 2)
    pair = (z[:, :, 0] + z[:, :, 1])[:, :, None].repeat(2, 2).reshape(M, -1)
    off = np.abs(G.host_f64(Y) - G.host_f64(R))
    assert (off <= 2.0 ** -8 * (pair + np.abs(G.host_f64(Y)) + np.abs(G.host_f64(R))) + 1e-4).all()


def test_position_outside_the_tables():
    """Status bit 0x2; that token passes through bit by bit, infinities and all."""
    import lora_linear_fine_b200 as L
    import torch
    Q, K, _ = _case(4, 2, 1, 64, 32, 8, 1)
    Q[1, 0], Q[3, 5] = float("inf"), float("nan")
    pos = torch.tensor([0, 8, 7, -1], dtype=torch.int32, device="cuda")
    cos, sin = L.rotary_tables(8, 32)
    ws = L.Workspace(256)
    Yq, Yk = L.rotary(Q, K, pos, cos, sin, 64, workspace=ws)
    assert ws.status() == 2
    for x, y in ((Q, Yq), (K, Yk)):
        assert torch.equal(x.view(torch.int16)[[1, 3]], y.view(torch.int16)[[1, 3]])
        assert torch.equal(x[0], y[0]) and not torch.equal(x[2], y[2])


def test_no_tokens_graph_and_stream():
    import lora_linear_fine_b200 as L
    import torch
    cos, sin = L.rotary_tables(64, 64)
    none = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    Yq, Yk = L.rotary(none, none, torch.empty(0, dtype=torch.int32, device="cuda"), cos, sin, 64)
    assert Yq.shape == Yk.shape == (0, 128)
    Q, K, pos = _case(500, 6, 2, 64, 64, 64, 2)
    ws = L.Workspace(256)
    Yq, Yk = L.rotary(Q, K, pos, cos, sin, 64, workspace=ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a, b = L.rotary(Q, K, pos, cos, sin, 64, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(a, Yq) and torch.equal(b, Yk)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = L.rotary(Q, K, pos, cos, sin, 64, workspace=ws)
    pos.copy_(63 - pos)
    graph.replay()
    c, d = L.rotary(Q, K, pos, cos, sin, 64, workspace=ws)
    assert torch.equal(a, c) and torch.equal(b, d) and not torch.equal(a, Yq)


def test_offsets_past_32_bits():
    import lora_linear_fine_b200 as L
    import torch
    hd, heads = 128, 64
    M = (1 << 31) // (hd * heads) + 100
    Q = torch.zeros(M, heads * hd, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(3, heads * hd, device="cuda").bfloat16()
    Q[-3:] = tail
    pos = torch.zeros(M, dtype=torch.int32, device="cuda")
    pos[-3:] = torch.tensor([5, 60, 31], dtype=torch.int32)
    cos, sin = L.rotary_tables(64, hd)
    Y, _ = L.rotary(Q, None, pos, cos, sin, hd, inplace=True)
    y, _ = L.rotary(tail, None, pos[-3:].contiguous(), cos, sin, hd)
    assert torch.equal(Y[-3:], y)
