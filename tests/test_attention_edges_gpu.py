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
@pytest.mark.parametrize("cap", [0.0, 2.0, 30.0, 70.0, 1e6])
@pytest.mark.parametrize("D", [64, 128])
def test_documents_do_not_touch_each_other_under_a_cap(D, cap, bias):
    """Large values, infinities and NaN in one document leave the other
    documents' bits, whichever way they make the tanh be taken or the running
    reference move."""
    import torch
    lens = [100, 60, 200]

    def poison(Q, K, V, dO):
        Q[105], K[101], K[120], V[130] = (float("nan"), float("-inf"), float("inf"), float("nan"))
        Q[112] = 1e20

    def large(Q, K, V, dO):
        Q[100:160] *= 64.0
        K[100:160] *= 64.0

    for causal in (True, False):
        kw = dict(seed=16, causal=causal, cap=cap, slopes=[0.25, -0.5, 0.0, 0.01] if bias else None)
        clean, _, _, _ = _run(lens, 40, 4, 2, D, **kw)
        for edit in (poison, large):
            out, _, _, _ = _run(lens, 40, 4, 2, D, edit=edit, **kw)
            for name in clean:
                assert torch.equal(out[name][:100], clean[name][:100]), name
                assert torch.equal(out[name][160:], clean[name][160:]), name


@pytest.mark.parametrize("cap", [1e4, 1e5, 1e6, 1e9, 1e25, 3e38])
@pytest.mark.parametrize("D", [64, 128])
def test_caps_far_above_the_scores(D, cap):
    _within_bounds([200, 77, 260], 4, 2, D, cap=cap, seed=31)
    _within_bounds([200, 77, 260], 4, 2, D, cap=cap, seed=32, slopes=[0.5, -0.01, 0.0, 1.0])


@pytest.mark.parametrize("cap", [1e-3, 1.0, 55.0, 1e4, 1e7])
@pytest.mark.parametrize("down", [-20, 3, 16, 18, 30, 50])
@pytest.mark.parametrize("D", [64, 128])
def test_capped_score_of_one_key(D, down, cap):
    """lse of a row with one key is its score cap tanh(y), for |y| from about
    2^-20 to 2^4 and scale / cap = 2^-down: to half steps of the sum of the
    products and some sixteen of the result (near y = 0.4, where the tanh by the
    exponential takes over, 2^-22 of it is twelve)."""
    import lora_linear_fine_b200 as L
    import torch
    n = 48
    Q, K, V, dO = (t.cuda() for t in _inputs(n, 2, 2, D, 33))
    Q *= (2.0 ** (torch.linspace(-20, 4, n).floor() + down - 3)).bfloat16().cuda()[:, None]
    plan = L.AttentionPlan(torch.arange(n + 1, dtype=torch.int32, device="cuda"), n)
    c = float(np.float32(cap))
    kw = dict(scale=c * 2.0 ** -down, softcap=c)
    o, lse = L.attention(Q, K, V, plan, 2, 2, **kw)
    dQ, dK, dV = L.attention_backward(dO, Q, K, V, o, lse, plan, 2, 2, **kw)
    terms = kw["scale"] * G.host_f64(Q).reshape(n, 2, D) * G.host_f64(K).reshape(n, 2, D)
    z = c * np.tanh(terms.sum(-1) / c)
    off = np.abs(G.host_f64(lse) - z)
    assert (off <= 2.0 ** -24 * (D * np.abs(terms).sum(-1) + 16 * np.abs(z))).all(), (off / np.abs(z)).max()
    assert not dQ.any() and not dK.any()
    # p and its sum are 2^e, e what the reference is off by: p is rounded to bf16 and then the quotient
    near = lambda got, want, rows: (np.abs(G.host_f64(got[rows]) - G.host_f64(want[rows])) <=
                                    2.0 ** -7 * (1 + 2.0 ** -8) * np.abs(G.host_f64(want[rows]))).all()
    assert near(o, V, slice(None))
    # the backward's p is exp(z - lse): within 2^-15 of 1 where z is below 2^6
    assert near(dV, dO, np.abs(z).max(1) < 64)


@pytest.mark.parametrize("down", [3, 18, 30])
@pytest.mark.parametrize("cap", [1.0, 32.0])
def test_gradients_of_capped_scores(cap, down):
    """Documents of two equal keys, whose p is 1/2 whatever their score: dK
    carries the cap's derivative, for scores of 2^-6 to twice the cap and
    scale / cap = 2^-down."""
    import lora_linear_fine_b200 as L
    import torch
    D, n = 64, 40
    Q, K, V, dO = (t.cuda() for t in _inputs(2 * n, 2, 1, D, 34))
    K[1::2] = K[::2]
    Q *= (2.0 ** (torch.linspace(-6, 1, n).floor() + down - 3)).bfloat16().cuda().repeat_interleave(2)[:, None]
    starts = np.arange(0, 2 * n + 1, 2)
    plan = L.AttentionPlan(torch.from_numpy(starts).int().cuda(), 2 * n, causal=False)
    kw = dict(scale=cap * 2.0 ** -down, softcap=cap)
    o, lse = L.attention(Q, K, V, plan, 2, 1, **kw)
    got = dict(zip(("dQ", "dK", "dV"), L.attention_backward(dO, Q, K, V, o, lse, plan, 2, 1, **kw)), O=o, lse=lse)
    # scores up to 2^5: 2^-12 in place of the 2^-14 for scores up to 2^3
    ref = O.attention(*(G.host_f64(t) for t in (Q, K, V)), starts, 2, 1, causal=False, dO=G.host_f64(dO), bounds=True,
                      fp=2.0 ** -12, **kw)
    for name, t in got.items():
        t = G.host_f64(t)
        assert np.isfinite(t).all(), name
        assert (np.abs(t - ref[name]) <= ref["tol"][name] + 1e-30).all(), name


@pytest.mark.parametrize("kw", [dict(), dict(cap=30.0), dict(slopes=[0.25, 0.0])], ids=["plain", "cap", "bias"])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_in_a_key(D, kw):
    """A key of NaN, at every column of a group of eight: NaN in O, lse and dQ
    of the rows that see it (by whatever form their exponentials are taken), no
    change to the others; NaN in dV of every key that those rows see."""
    import torch
    for lens in ([16], [200]):
        n = lens[0]
        clean, _, _, _ = _run(lens, 0, 2, 1, D, seed=35, **kw)
        for j in list(range(8)) + ([133] if n > 133 else []):
            def edit(Q, K, V, dO):
                K[j] = float("nan")

            out, _, _, _ = _run(lens, 0, 2, 1, D, seed=35, edit=edit, **kw)
            for name in ("O", "lse", "dQ"):
                assert torch.isnan(out[name][j:]).all(), (name, j)
            for name in ("O", "lse"):
                assert torch.equal(out[name][:j], clean[name][:j]), (name, j)
            assert torch.isnan(out["dV"]).all(), j


@pytest.mark.parametrize("made", [True, False])
def test_plan_of_another_mask(made):
    """A causal plan with a call for whole documents, or the reverse: status bit
    0x2 and nothing computed, forward and backward."""
    import lora_linear_fine_b200 as L
    import torch
    starts = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    Q, K, V, dO = (t.cuda() for t in _inputs(64, 2, 2, 64, 0))
    st = torch.cuda.current_stream().cuda_stream
    desc = L.make_attn_desc(64, 1, 2, 2, 64, causal=not made)
    plan = L.AttentionPlan(starts, 64, causal=made)
    o, lse = torch.full_like(Q, 3.0), torch.full((64, 2), 3.0, device="cuda")
    assert L.lora_linear_attn_fwd(desc, plan.buf.data_ptr(), plan.nbytes, Q.data_ptr(), K.data_ptr(), V.data_ptr(),
                                  None, o.data_ptr(), lse.data_ptr(), st) == 0
    assert torch.all(o == 3.0) and torch.all(lse == 3.0) and plan.status() == 2
    plan = L.AttentionPlan(starts, 64, causal=made)
    ws = L.Workspace(L.lora_linear_attn_workspace_size(desc))
    g = [torch.full_like(Q, 3.0) for _ in range(3)]
    assert L.lora_linear_attn_bwd(desc, plan.buf.data_ptr(), plan.nbytes, dO.data_ptr(), Q.data_ptr(), K.data_ptr(),
                                  V.data_ptr(), o.data_ptr(), lse.data_ptr(), None, *(t.data_ptr() for t in g),
                                  ws.buf.data_ptr(), ws.nbytes, st) == 0
    assert all(torch.all(t == 3.0) for t in g) and plan.status() == 2
