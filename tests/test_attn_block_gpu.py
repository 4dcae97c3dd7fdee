"""Layer norm, LoRA projections, rotary positions and attention over packed
documents as one attention block, forward and backward, against the same block
in fp64 with gradients by differentiation."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _lin(x, W, A, B, s):
    return x @ W.T + s * (x @ A.T) @ B.T


@pytest.mark.parametrize("layout,rot,cap,bias", [("half", 64, 0.0, False), ("interleaved", 32, 30.0, True)])
@pytest.mark.parametrize("lens,pad", [([1], 0), ([100, 28], 0), ([130, 1, 0, 70, 45], 10)])
def test_block(lens, pad, layout, rot, cap, bias):
    import lora_linear_fine_b200 as L
    import torch
    H, Gk, D, d, r, s = 4, 2, 64, 256, 8, 2.0
    M = sum(lens) + pad
    gen = torch.Generator().manual_seed(sum(lens) + rot)
    n = lambda *z, by=1.0: (torch.randn(*z, generator=gen) * by).bfloat16().cuda()
    X, g, b, dO = n(M, d), 1 + n(d, by=0.1), n(d, by=0.1), n(M, H * D)
    outs = (H * D, Gk * D, Gk * D)
    Ws = [n(o, d, by=d ** -0.5) for o in outs]
    As = [n(r, d, by=d ** -0.5) for _ in outs]
    Bs = [n(o, r, by=r ** -0.5) for o in outs]
    starts = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(x) for x in lens + [pad]]).to(torch.int32).cuda()
    slopes = torch.tensor([0.25, 0.0625, 0.015625, 0.00390625], device="cuda") if bias else None
    kw = dict(heads=H, kv_heads=Gk, softcap=cap, slopes=slopes)

    plan = L.AttentionPlan(starts, M)
    cos, sin = L.rotary_tables(256, rot)
    ws = L.Workspace(256)
    Xn, mean, rstd = L.layer_norm(X, g, b)
    (q, Tq, _), (k, Tk, _), (v, Tv, _) = (L.forward(Xn, W, A, B, s) for W, A, B in zip(Ws, As, Bs))
    qr, kr = L.rotary(q, k, pos, cos, sin, D, layout, workspace=ws)
    O, lse = L.attention(qr, kr, v, plan, **kw)
    dqr, dkr, dv = L.attention_backward(dO, qr, kr, v, O, lse, plan, **kw)
    dq, dk = L.rotary(dqr, dkr, pos, cos, sin, D, layout, inverse=True, workspace=ws)
    parts = [L.backward(dy, Xn, W, A, B, s, T_save=T) for dy, W, A, B, T in zip((dq, dk, dv), Ws, As, Bs, (Tq, Tk, Tv))]
    dXn = sum(p[0].float() for p in parts)
    dX, dg, db = L.layer_norm_backward(dXn, X, g, mean, rstd)
    assert plan.status() == 0 and ws.status() == 0

    x, gg, bb = (t.double().requires_grad_() for t in (X, g, b))
    AA, BB = ([t.double().requires_grad_() for t in ts] for ts in (As, Bs))
    mu = x.mean(1, keepdim=True)
    xn = (x - mu) / ((x - mu).pow(2).mean(1, keepdim=True) + 1e-5).sqrt() * gg + bb
    y = [_lin(xn, W.double(), A, B, s) for W, A, B in zip(Ws, AA, BB)]
    c, sn = cos.double()[pos.long()][:, None], sin.double()[pos.long()][:, None]

    def turned(t):
        t = t.view(M, -1, D)
        i = torch.arange(rot // 2, device="cuda")
        ia, ib = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        z = t.clone()
        z[..., ia], z[..., ib] = t[..., ia] * c - t[..., ib] * sn, t[..., ib] * c + t[..., ia] * sn
        return z

    Q, K, V = turned(y[0]), turned(y[1]).repeat_interleave(H // Gk, 1), y[2].view(M, Gk, D).repeat_interleave(H // Gk, 1)
    rows = []
    at = starts.tolist()
    for a, e in zip(at, at[1:]):
        z = torch.einsum("ihd,jhd->hij", Q[a:e], K[a:e]) * D ** -0.5
        if cap:
            z = cap * torch.tanh(z / cap)
        i = torch.arange(e - a, device="cuda", dtype=torch.float64)
        if bias:
            z = z - slopes.double()[:, None, None] * (i[:, None] - i).abs()
        z = z.masked_fill(i[:, None] < i, float("-inf"))
        rows.append(torch.einsum("hij,jhd->ihd", torch.softmax(z, -1), V[a:e]))
    rows.append(torch.zeros(pad, H, D, dtype=torch.float64, device="cuda"))
    want = torch.cat(rows).reshape(M, -1)
    grads = torch.autograd.grad(want, [x, gg, bb] + AA + BB, dO.double())
    got = [O, dX, dg, db] + [p[1] for p in parts] + [p[2] for p in parts]
    names = ["O", "dX", "dg", "db", "dAq", "dAk", "dAv", "dBq", "dBk", "dBv"]
    # some ten roundings to bf16 lie one behind the other (relative rms 2^-9.3
    # each: 2^-7.6 together); scores of a few units multiply what reaches them
    for name, a, w in zip(names, got, [want.detach(), *grads]):
        off, size = (a.double() - w).norm().item(), w.norm().item()
        if sum(lens) == 1 and name in ("dAq", "dAk", "dBq", "dBk"):
            assert off == 0.0, name                      # one key: the scores have no gradient
        else:
            assert off <= 2.0 ** -5 * size, f"{name}: {off:.3g} of {size:.3g}"
