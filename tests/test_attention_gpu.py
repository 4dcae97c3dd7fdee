"""Attention over packed documents against its fp64 statement, with the
element bounds that oracle/attn_block_oracle.py derives from the roundings to
bf16 (p, ds, the outputs) and the fp32 arithmetic."""
import numpy as np
import pytest

from oracle import attn_block_oracle as O
from tests import gpu_cases as G

pytestmark = pytest.mark.gpu


def _starts(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def _inputs(M, H, Gk, D, seed, spread=1.0):
    import torch
    gen = torch.Generator().manual_seed(seed)
    n = lambda h, s=1.0: (s * torch.randn(M, h * D, generator=gen)).bfloat16()
    return n(H, spread), n(Gk, spread), n(Gk), n(H)


def _run(lens, pad, H, Gk, D, causal=True, prefix=None, cap=0.0, slopes=None, seed=0, spread=1.0, scale=None,
         edit=None):
    """One forward and backward; (outputs, inputs, plan, keyword arguments)."""
    import lora_linear_fine_b200 as L
    import torch
    M = int(sum(lens)) + pad
    x = [t.cuda() for t in _inputs(M, H, Gk, D, seed, spread)]
    if edit:
        edit(*x)
    starts = torch.from_numpy(_starts(lens)).cuda()
    pre = None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device="cuda")
    plan = L.AttentionPlan(starts, M, prefix_len=pre, causal=causal)
    kw = dict(heads=H, kv_heads=Gk, scale=scale, softcap=cap,
              slopes=None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device="cuda"))
    Q, K, V, dO = x
    o, lse = L.attention(Q, K, V, plan, **kw)
    dQ, dK, dV = L.attention_backward(dO, Q, K, V, o, lse, plan, **kw)
    assert plan.status() == 0
    return {"O": o, "lse": lse, "dQ": dQ, "dK": dK, "dV": dV}, x, plan, kw


def _check(lens, pad, H, Gk, D, **c):
    out, x, _, _ = _run(lens, pad, H, Gk, D, **c)
    Q, K, V, dO = (G.host_f64(t) for t in x)
    ref = O.attention(Q, K, V, _starts(lens), H, Gk, prefix=c.get("prefix"), causal=c.get("causal", True),
                      scale=c.get("scale"), softcap=c.get("cap", 0.0),
                      slopes=None if c.get("slopes") is None else np.array(c["slopes"], dtype=np.float32).astype(float),
                      dO=dO, bounds=True)
    for name, got in out.items():
        got, want, tol = G.host_f64(got), ref[name], ref["tol"][name]
        gone = np.isneginf(want)
        assert np.array_equal(gone, np.isneginf(got)), name
        off = np.where(gone, 0.0, np.abs(np.where(gone, 0, got) - np.where(gone, 0, want)))
        assert np.isfinite(off).all(), f"{name}: {np.count_nonzero(~np.isfinite(off))} values are not finite"
        worst = (off / (tol + 1e-30)).max() if off.size else 0.0
        assert worst <= 1.0, f"{name}: {worst:.3g} times its bound"


LENS = [[1], [2], [96], [127], [128], [129], [255], [256], [257], [300, 1, 0, 64, 130], [1] * 20, [500], [385, 260]]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", LENS, ids=lambda v: "-".join(map(str, v[:5])))
def test_causal(lens, D):
    _check(lens, 0, 4, 2, D, seed=sum(lens) + D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Gk", [(1, 1), (3, 3), (8, 1), (6, 2)])
def test_heads(H, Gk, D):
    _check([150, 3], 5, H, Gk, D, seed=H)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[1], [130, 256, 70], [400]], ids=lambda v: "-".join(map(str, v)))
def test_whole_documents(lens, D):
    _check(lens, 3, 4, 2, D, causal=False, seed=7)


@pytest.mark.parametrize("D", [64, 128])
def test_prefix(D):
    _check([1, 200, 129, 300, 0, 390], 1, 4, 2, D, prefix=[1, 0, 129, 140, 0, 270], seed=8)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [0.5, 5.0, 50.0])
def test_softcap(cap, D):
    _check([200, 77, 260], 9, 4, 2, D, cap=cap, seed=9)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,H,Gk", [([200, 77, 260], 4, 2), ([500], 2, 2), ([1500, 1500], 16, 16)])
def test_warps_at_uneven_speed(lens, H, Gk, D):
    """A cap whose tanh takes the long way in some warps and the short one in
    others, so that the warps of a tile drift apart: the same bits every time."""
    import torch
    cap = 1.0

    def edit(Q, K, V, dO):
        Q[::97] *= 4.0
        Q[1::3] *= 0.05

    first, (Q, K, V, dO), plan, kw = _run(lens, 0, H, Gk, D, cap=cap, seed=23, edit=edit)
    if sum(lens) < 1000:
        ref = O.attention(*(G.host_f64(t) for t in (Q, K, V)), _starts(lens), H, Gk, softcap=cap, dO=G.host_f64(dO))
        for name in first:
            off = np.linalg.norm(G.host_f64(first[name]) - ref[name]) / np.linalg.norm(ref[name])
            assert off <= 2.0 ** -7, f"{name}: {off:.3g}"      # roundings of p, ds, the output: 2^-9 rms each
    import lora_linear_fine_b200 as L
    for _ in range(15):
        o, lse = L.attention(Q, K, V, plan, **kw)
        got = (o, lse) + L.attention_backward(dO, Q, K, V, o, lse, plan, **kw)
        assert all(torch.equal(a, b) for a, b in zip(first.values(), got))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("cap", [0.0, 10.0])
@pytest.mark.parametrize("D", [64, 128])
def test_distance_bias(D, cap, causal):
    _check([200, 77, 260], 0, 4, 2, D, slopes=[0.5, 0.0, 2.0 ** -8, 1.0], cap=cap, causal=causal, seed=10)


@pytest.mark.parametrize("D", [64, 128])
def test_prefix_with_bias_and_cap(D):
    _check([300, 150], 0, 2, 2, D, prefix=[133, 150], slopes=[0.25, 0.03], cap=8.0, seed=11)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("cap", [0.0, 7.0])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_see_one_key(D, cap, causal):
    """The softmax of one score does not depend on it: dQ is zero exactly, and so
    is dK of a document of one row; lse is the score."""
    lens = [1, 1, 5, 1, 130, 1]
    out, (Q, K, V, dO), _, _ = _run(lens, 2, 4, 2, D, cap=cap, causal=causal, seed=19)
    one = [0, 1, 7, 138]
    first = [2, 8]
    assert not out["dQ"][one + (first if causal else [])].any() and not out["dK"][one].any()
    z = (Q[one].double().view(4, 4, D) * K[one].double().view(4, 2, D).repeat_interleave(2, 1)).sum(-1) * D ** -0.5
    z = cap * np.tanh(G.host_f64(z) / cap) if cap else G.host_f64(z)
    # a handful of fp32 roundings of a sum of D terms of a few units
    assert np.abs(G.host_f64(out["lse"][one]) - z).max() <= 2.0 ** -20 * (4 + np.abs(z).max())
    # p is 1 where the reference is the row's maximum.  Under a cap it is not, and
    # p / l = 1 with p rounded to bf16 (half a step, 2^-8) times V is rounded once
    # more: (1 + 2^-8)^2 - 1 <= 2^-7 (1 + 2^-9)
    got, want = (G.host_f64(t) for t in (out["O"][one].view(4, 4, D), V[one].view(4, 2, D).repeat_interleave(2, 1)))
    assert (np.abs(got - want) <= (2.0 ** -7 * (1 + 2.0 ** -9) if cap else 0.0) * np.abs(want)).all()


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("cap", [2.0, 50.0])
@pytest.mark.parametrize("D", [64, 128])
def test_one_key_with_a_cap(D, cap, bias):
    """One key a row and scores near zero: O is V, and lse is the score to the
    precision of the score, not of a sum of exponentials near one."""
    lens = [1] * 9
    kw = dict(slopes=[0.25, 0.01]) if bias else {}
    out, (Q, K, V, _), _, _ = _run(lens, 0, 2, 1, D, cap=cap, scale=0.002, seed=21, **kw)
    # p is 1 but for 2^-16, which bf16 rounds away in p and again in the quotient
    want = G.host_f64(V.view(9, 1, D).expand(9, 2, D))
    assert np.array_equal(G.host_f64(out["O"].view(9, 2, D)), want)
    terms = G.host_f64(Q).reshape(9, 2, D) * G.host_f64(K).reshape(9, 1, D) * 0.002
    z = cap * np.tanh(terms.sum(-1) / cap)
    # the sum of D products in fp32, and some ten roundings of the result
    tol = 2.0 ** -24 * (D * np.abs(terms).sum(-1) + 16 * np.abs(z))
    assert (np.abs(G.host_f64(out["lse"]).reshape(9, 2) - z) <= tol).all()


def test_gradients_of_short_documents():
    """Rows with a few keys: delta is not the one of the rounded O, so dQ and dK
    stay within the roundings of ds (2^-9 rms each) and of the output."""
    import torch
    lens = [2] * 9 + [3] * 7 + [4, 7, 11]
    out, (Q, K, V, dO), _, _ = _run(lens, 0, 4, 2, 128, cap=20.0, seed=20)
    ref = O.attention(*(G.host_f64(t) for t in (Q, K, V)), _starts(lens), 4, 2, softcap=20.0, dO=G.host_f64(dO))
    for name in ("dQ", "dK", "dV"):
        off = np.linalg.norm(G.host_f64(out[name]) - ref[name]) / np.linalg.norm(ref[name])
        assert off <= 2.0 ** -8, f"{name}: {off:.3g}"


def test_scale_and_large_scores():
    """Scores of a few tens, where one key takes almost all of a row."""
    _check([260, 100], 0, 2, 1, 64, scale=0.02, seed=12)
    _check([260, 100], 0, 2, 1, 128, spread=1.6, seed=13)


@pytest.mark.parametrize("kw", [dict(), dict(slopes=[0.01, -0.005]), dict(cap=100.0), dict(cap=100.0, slopes=[0.02, -0.01])],
                         ids=["plain", "bias", "cap", "both"])
@pytest.mark.parametrize("D", [64, 128])
def test_far_keys_dominate(D, kw):
    """Scores that rise by tens from the nearest tile to the far ones: the
    running reference moves, for some rows and not for others."""
    def edit(Q, K, V, dO):
        K[:100] *= 6.0
        K[200:260] *= 3.0

    lens = [600, 90]
    out, x, _, _ = _run(lens, 0, 2, 1, D, seed=21, edit=edit, cap=kw.get("cap", 0.0), slopes=kw.get("slopes"))
    Q, K, V, dO = (G.host_f64(t) for t in x)
    slopes = None if kw.get("slopes") is None else np.array(kw["slopes"], dtype=np.float32).astype(float)
    ref = O.attention(Q, K, V, _starts(lens), 2, 1, softcap=kw.get("cap", 0.0), slopes=slopes, dO=dO)
    # scores up to 2^6: their fp32 error 2^-24 2^6 2^2 turns into a relative
    # 2^-16 of p; the roundings of p, ds and the outputs (2^-9 rms) remain
    for name in ("O", "dQ", "dK", "dV"):
        off = np.linalg.norm(G.host_f64(out[name]) - ref[name]) / np.linalg.norm(ref[name])
        assert off <= 2.0 ** -7, f"{name}: {off:.3g}"
    assert np.abs(G.host_f64(out["lse"]) - ref["lse"]).max() <= 2.0 ** -14


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("cap", [0.0, 10.0, 70.0])
def test_rising_bias(cap, causal):
    """Negative slopes favour the far keys."""
    _check([200, 77, 260], 0, 4, 2, 64, slopes=[-0.5, 0.0, -2.0 ** -8, 0.25], cap=cap, causal=causal, seed=22)


def test_rows_behind_the_last_document():
    """Zeros and -inf, whatever the inputs hold there; no document changes."""
    import torch

    def poison(Q, K, V, dO):
        for t, v in ((Q, float("nan")), (K, float("inf")), (V, float("nan")), (dO, float("-inf"))):
            t[330:] = v

    for D in (64, 128):
        clean, _, _, _ = _run([200, 130], 170, 4, 2, D, seed=14)
        out, _, _, _ = _run([200, 130], 170, 4, 2, D, seed=14, edit=poison)
        for name in clean:
            assert torch.equal(out[name], clean[name]), name
            rest = out[name][330:]
            assert torch.isneginf(rest).all() if name == "lse" else not rest.any()


def test_only_rows_behind():
    import torch
    for lens in ([], [0, 0]):
        out, _, _, _ = _run(lens, 140, 2, 1, 64, seed=15)
        assert torch.isneginf(out["lse"]).all() and not any(out[n].any() for n in ("O", "dQ", "dK", "dV"))


def test_no_rows():
    out, _, _, _ = _run([], 0, 2, 1, 128)
    assert out["O"].shape == (0, 256) and out["dK"].shape == (0, 128)


def test_documents_do_not_touch_each_other():
    """NaN and infinities in one document leave the other documents' bits."""
    import torch
    lens = [100, 60, 200]

    def poison(Q, K, V, dO):
        Q[110], K[120], V[130], V[150], dO[140] = (float("nan"), float("inf"), float("nan"), float("-inf"), float("nan"))

    for D in (64, 128):
        for causal in (True, False):
            clean, _, _, _ = _run(lens, 40, 4, 2, D, seed=16, causal=causal)
            out, _, _, _ = _run(lens, 40, 4, 2, D, seed=16, causal=causal, edit=poison)
            for name in clean:
                assert torch.equal(out[name][:100], clean[name][:100]), name
                assert torch.equal(out[name][160:], clean[name][160:]), name
                assert not torch.isfinite(out[name][100:160].float()).all()


def test_same_bits_graph_and_streams():
    """The same bits again, on two streams at once over one plan, and from a
    captured step replayed on new inputs and a new plan of the same sizes."""
    import lora_linear_fine_b200 as L
    import torch
    lens = [300, 45, 200]
    out, (Q, K, V, dO), plan, kw = _run(lens, 11, 4, 2, 128, seed=17)
    args = (Q, K, V)

    def step(ws, stream=None):
        o, lse = L.attention(*args, plan, **kw, stream=stream)
        return (o, lse) + L.attention_backward(dO, *args, o, lse, plan, **kw, workspace=ws, stream=stream)

    desc = L.make_attn_desc(Q.shape[0], 3, 4, 2, 128)
    ws = [L.Workspace(L.lora_linear_attn_workspace_size(desc)) for _ in range(3)]
    first = tuple(out.values())
    assert all(torch.equal(a, b) for a, b in zip(first, step(ws[0])))
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [step(ws[k], side[k]) for k in (0, 1)]
    for k in (0, 1):
        side[k].synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, got[k]))
    starts = torch.from_numpy(_starts(lens)).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan = L.AttentionPlan(starts, Q.shape[0])
        held = step(ws[2])
    starts.copy_(torch.tensor([0, 10, 400, 540], dtype=torch.int32))
    V.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    held = [t.clone() for t in held]
    plan = L.AttentionPlan(starts, Q.shape[0])
    assert all(torch.equal(a, b) for a, b in zip(held, step(ws[0])))


@pytest.mark.parametrize("starts,prefix", [([1, 5], None), ([0, 9, 5], None), ([0, 65], None), ([0, -1, 5], None),
                                           ([0, 10], [11]), ([0, 10], [-1])])
def test_bad_documents(starts, prefix):
    """Status bit 0x2, and nothing is computed."""
    import lora_linear_fine_b200 as L
    import torch
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    plan = L.AttentionPlan(i32(starts), 64, prefix_len=None if prefix is None else i32(prefix))
    assert plan.status() == 2
    Q, K, V, dO = (t.cuda() for t in _inputs(64, 2, 2, 64, 0))
    o, lse = torch.full_like(Q, 3.0), torch.full((64, 2), 3.0, device="cuda")
    desc = L.make_attn_desc(64, len(starts) - 1, 2, 2, 64)
    assert L.lora_linear_attn_fwd(desc, plan.buf.data_ptr(), plan.nbytes, Q.data_ptr(), K.data_ptr(), V.data_ptr(),
                                  None, o.data_ptr(), lse.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.all(o == 3.0) and torch.all(lse == 3.0)


def test_plan_of_other_sizes():
    """A plan made for fewer rows than the call has: refused by the torch
    functions, status bit 0x2 and nothing computed through the C entry point."""
    import lora_linear_fine_b200 as L
    import torch
    starts = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    plan = L.AttentionPlan(starts, 64)
    Q, K, V, _ = (t.cuda() for t in _inputs(50, 2, 2, 64, 0))
    with pytest.raises(L.LoraError):
        L.attention(Q, K, V, plan, 2, 2)
    with pytest.raises(L.LoraError):
        L.attention(Q, K[:, :64], V, plan, 2, 2)
    o, lse = torch.full_like(Q, 3.0), torch.full((50, 2), 3.0, device="cuda")
    desc = L.make_attn_desc(50, 1, 2, 2, 64)
    assert L.lora_linear_attn_fwd(desc, plan.buf.data_ptr(), plan.nbytes, Q.data_ptr(), K.data_ptr(), V.data_ptr(),
                                  None, o.data_ptr(), lse.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.all(o == 3.0) and plan.status() == 2


def test_long_document():
    """A document of many tiles, some rows and keys compared."""
    import torch
    n, D = 3001, 128
    out, x, _, _ = _run([n], 0, 2, 1, D, seed=18)
    Q, K, V, dO = (t.double() for t in x)
    k, v = K.requires_grad_(), V.requires_grad_()
    Q.requires_grad_()
    q = Q.view(n, 2, D).transpose(0, 1)
    z = (q @ k.T) * D ** -0.5
    z = z.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), float("-inf"))
    o = (torch.softmax(z, -1) @ v).transpose(0, 1).reshape(n, -1)
    o.backward(dO)
    # independent roundings of relative rms 2^-9.8 in p (or ds) and the output
    # keep the whole within 2^-8 of its norm
    for name, want in (("O", o), ("dQ", Q.grad), ("dK", k.grad), ("dV", v.grad)):
        got = out[name].double()
        assert torch.isfinite(got).all()
        assert (got - want).norm() <= 2.0 ** -8 * want.norm(), name


def test_offsets_past_32_bits():
    """Documents behind 2^31 elements of Q: the same as on their own (dK and dV
    of the small batch are summed in parts: fp32 sums in another order, then one
    rounding each, so at most one bf16 step, 2^-7, apart)."""
    import lora_linear_fine_b200 as L
    import torch
    H, Gk, D = 64, 8, 128
    M = (1 << 31) // (H * D) + 700
    gen = torch.Generator(device="cuda").manual_seed(1)
    Q = torch.zeros(M, H * D, dtype=torch.bfloat16, device="cuda")
    K, V = (torch.zeros(M, Gk * D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    small = [torch.randn(400, h * D, generator=gen, device="cuda").bfloat16() for h in (H, Gk, Gk)]
    for t, s in zip((Q, K, V), small):
        t[-400:] = s
    starts = list(range(0, M - 400, 1000))[:-1] + [M - 400, M - 150, M]
    plan = L.AttentionPlan(torch.tensor(starts, dtype=torch.int32, device="cuda"), M)
    o, lse = L.attention(Q, K, V, plan, H, Gk)
    p2 = L.AttentionPlan(torch.tensor([0, 250, 400], dtype=torch.int32, device="cuda"), 400)
    o2, lse2 = L.attention(*small, p2, H, Gk)
    assert torch.equal(o[-400:], o2) and torch.equal(lse[-400:], lse2)
    dO = Q.clone()
    g = L.attention_backward(dO, Q, K, V, o, lse, plan, H, Gk)
    del dO
    g2 = L.attention_backward(small[0].clone(), *small, o2, lse2, p2, H, Gk)
    assert torch.equal(g[0][-400:], g2[0])
    for a, b in zip(g[1:], g2[1:]):
        a, b = a[-400:].float(), b.float()
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -16 * b.abs().max()).all()
