"""The fp64 statements of layer norm, rotary positions and attention
(oracle/attn_block_oracle.py) held to facts that do not come from their code:
hand values, and gradients against central differences."""
import numpy as np
import pytest

from oracle import attn_block_oracle as O


def _differences(f, x, g, at, h=1e-5):
    """d <f(x), g> / d x at the flat indexes `at`."""
    got = []
    for i in at:
        d = np.zeros(x.size)
        d[i] = h
        d = d.reshape(x.shape)
        got.append(((f(x + d) - f(x - d)) * g).sum() / (2 * h))
    return np.array(got)


def test_layer_norm_by_hand():
    Y, mean, rstd = O.layer_norm(np.array([[1.0, 3.0], [2.0, 2.0]]), np.array([2.0, 1.0]), np.array([0.5, 0.0]), 0.25)
    assert np.allclose(mean, [2.0, 2.0])
    assert np.allclose(rstd, [1 / np.sqrt(1.25), 2.0])
    assert np.allclose(Y, [[0.5 - 2 / np.sqrt(1.25), 1 / np.sqrt(1.25)], [0.5, 0.0]])


def test_layer_norm_gradient():
    r = np.random.default_rng(0)
    X, g, b, dY = r.standard_normal((3, 8)), r.standard_normal(8), r.standard_normal(8), r.standard_normal((3, 8))
    dX, dg, db = O.layer_norm_backward(dY, X, g, 1e-3)
    assert np.allclose(dX.ravel(), _differences(lambda x: O.layer_norm(x, g, b, 1e-3)[0], X, dY, range(24)), atol=1e-7)
    assert np.allclose(dg, _differences(lambda w: O.layer_norm(X, w, b, 1e-3)[0], g, dY, range(8)), atol=1e-7)
    assert np.allclose(db, _differences(lambda w: O.layer_norm(X, g, w, 1e-3)[0], b, dY, range(8)), atol=1e-7)


def test_rotary_by_hand():
    """A quarter turn of the first pair, none of the second; the feature past the rotated part stays."""
    cos, sin = np.array([[1.0, 1.0], [0.0, 1.0]]), np.array([[0.0, 0.0], [1.0, 0.0]])
    x = np.array([[1.0, 2.0, 3.0, 4.0, 9.0]])
    assert np.allclose(O.rotary(x, np.array([1]), cos, sin, 5, "half"), [[-3.0, 2.0, 1.0, 4.0, 9.0]])
    assert np.allclose(O.rotary(x, np.array([1]), cos, sin, 5, "interleaved"), [[-2.0, 1.0, 3.0, 4.0, 9.0]])
    assert np.allclose(O.rotary(x, np.array([0]), cos, sin, 5, "half"), x)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_inverse_is_the_adjoint(layout):
    r = np.random.default_rng(1)
    cos, sin = O.rotary_tables(9, 16, amplitude=1.3)
    pos = r.integers(0, 9, 5)
    x, y = r.standard_normal((5, 2 * 24)), r.standard_normal((5, 2 * 24))
    f = O.rotary(x, pos, cos, sin, 24, layout)
    b = O.rotary(y, pos, cos, sin, 24, layout, inverse=True)
    assert np.isclose((f * y).sum(), (x * b).sum())


def test_rotary_scalings_at_their_ends():
    f = O.rotary_frequencies(64)
    assert np.allclose(O.rotary_frequencies(64, scaling="linear", factor=4.0), f / 4)
    n = O.rotary_frequencies(64, scaling="ntk", factor=4.0)
    assert np.isclose(n[0], 1.0) and np.isclose(n[-1], f[-1] / 4)      # the slowest pair is stretched by the factor
    for kind, high in (("wavelength", 4.0), ("ramp", 32.0)):
        w = O.rotary_frequencies(64, scaling=kind, factor=4.0, low=1.0, high=high, original=8192)
        assert np.isclose(w[0], f[0]) and np.isclose(w[-1], f[-1] / 4)
        assert np.all(w <= f * (1 + 1e-12)) and np.all(w >= f / 4 * (1 - 1e-12))


def test_attention_by_hand():
    """Two documents of one and two rows: a single key passes its value
    through; equal scores average the values."""
    Q, K = np.zeros((3, 2)), np.ones((3, 2))
    V = np.array([[1.0, 2.0], [3.0, 5.0], [7.0, 9.0]])
    r = O.attention(Q, K, V, [0, 1, 3], 1, 1)
    assert np.allclose(r["O"], [[1, 2], [3, 5], [5, 7]])
    assert np.allclose(r["lse"][:, 0], [0, 0, np.log(2)])
    r = O.attention(Q, K, V, [0, 1, 3], 1, 1, prefix=[0, 2])
    assert np.allclose(r["O"], [[1, 2], [5, 7], [5, 7]])
    r = O.attention(Q, K, V, [0, 1, 3], 1, 1, causal=False, slopes=np.array([np.log(2.0)]))
    assert np.allclose(r["O"][1], (2 * V[1] + V[2]) / 3)
    r = O.attention(Q, K, V, [0, 1], 1, 1)                      # the rows behind the last document
    assert np.all(r["O"][1:] == 0) and np.all(np.isneginf(r["lse"][1:]))


@pytest.mark.parametrize("causal,prefix,cap,bias", [(True, None, 0.0, False), (True, [2, 1], 2.0, True),
                                                    (False, None, 1.5, False)])
def test_attention_gradient(causal, prefix, cap, bias):
    r = np.random.default_rng(3)
    M, H, G, D, starts = 8, 4, 2, 4, [0, 5, 7]
    Q, K, V = (r.standard_normal((M, n * D)) for n in (H, G, G))
    dO = r.standard_normal((M, H * D))
    kw = dict(prefix=prefix, causal=causal, softcap=cap, slopes=np.array([0.5, 0.25, 0.1, 0.3]) if bias else None)
    res = O.attention(Q, K, V, starts, H, G, dO=dO, **kw)
    at = r.choice(M * G * D, 20, replace=False)
    for name, f, x in (("dQ", lambda x: O.attention(x, K, V, starts, H, G, **kw)["O"], Q),
                       ("dK", lambda x: O.attention(Q, x, V, starts, H, G, **kw)["O"], K),
                       ("dV", lambda x: O.attention(Q, K, x, starts, H, G, **kw)["O"], V)):
        assert np.allclose(res[name].ravel()[at], _differences(f, x, dO, at), atol=1e-7), name
