"""Attention where its scores leave the usual range: biases that rise with the
distance under a cap, caps far above the scores, NaN and infinities, neighbours
in a tile, plans of another mask."""
import numpy as np
import pytest

from oracle import attn_block_oracle as O
from tests import gpu_cases as G
from tests.test_attention_gpu import _inputs, _run, _starts

pytestmark = pytest.mark.gpu


def _within_bounds(lens, H, Gk, D, fp=2.0 ** -14, **c):
    """_run's outputs within the oracle's element bounds; softcap and slopes as
    the kernels hold them, in fp32."""
    out, x, _, _ = _run(lens, 0, H, Gk, D, **c)
    Q, K, V, dO = (G.host_f64(t) for t in x)
    f32 = lambda v: np.asarray(v, dtype=np.float32).astype(float)
    ref = O.attention(Q, K, V, _starts(lens), H, Gk, causal=c.get("causal", True), scale=c.get("scale"),
                      softcap=float(f32(c.get("cap", 0.0))), slopes=None if c.get("slopes") is None else f32(c["slopes"]),
                      dO=dO, bounds=True, fp=fp)
    for name, got in out.items():
        off = np.abs(G.host_f64(got) - ref[name])
        assert np.isfinite(off).all(), f"{name}: {np.count_nonzero(~np.isfinite(off))} values are not finite"
        worst = (off / (ref["tol"][name] + 1e-30)).max()
        assert worst <= 1.0, f"{name}: {worst:.3g} times its bound"


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("cap", [0.0, 5.0, 30.0, 70.0])
@pytest.mark.parametrize("D", [64, 128])
def test_steeply_rising_bias(D, cap, causal):
    """Negative slopes under a cap: keys that a row does not see, among them the
    columns past a short document, lie far above those that it sees.

    Scores reach 4 * 200, exponents of 2 up to 2^10.2: each rounding of one is
    half a step of 2^-13.8, and an exponent takes some five (the slope's product
    with log2 e, its product with the distance, the reference or lse and its
    change of base, the sum), which p turns into a relative 2^-11.9."""
    for k, lens in enumerate(([1], [5, 1, 127], [128, 2, 200])):
        _within_bounds(lens, 4, 2, D, fp=2.0 ** -11, cap=cap, slopes=[-1.0, -4.0, 0.5, -2.0], causal=causal, seed=30 + k)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("cap", [2.0, 30.0])
@pytest.mark.parametrize("D", [64, 128])
def test_documents_do_not_touch_each_other_under_a_cap(D, cap, bias):
    """Large values, infinities and NaN in one document leave the other
    documents' bits, whichever way they make the tanh be taken."""
    import torch
    lens = [100, 60, 200]

    def poison(Q, K, V, dO):
        Q[105], K[101], K[120], V[130] = (float("nan"), float("-inf"), float("inf"), float("nan"))
        Q[112] = 1e20

    def large(Q, K, V, dO):
        Q[100:160] *= 64.0
        K[100:160] *= 64.0

    for causal in (True, False):
        kw = dict(seed=16, causal=causal, cap=cap, slopes=[0.25, -0.02, 0.0, 0.01] if bias else None)
        clean, _, _, _ = _run(lens, 40, 4, 2, D, **kw)
        for edit in (poison, large):
            out, _, _, _ = _run(lens, 40, 4, 2, D, edit=edit, **kw)
            for name in clean:
                assert torch.equal(out[name][:100], clean[name][:100]), name
                assert torch.equal(out[name][160:], clean[name][160:]), name
