"""The operators around the attention of a packed batch, as they are measured:
layer norm (forward and backward), rotary positions (tables and rotation) and
masked attention over documents (forward and backward).

``run`` makes one pass of a case; ``own`` chooses between the plain form
(elementary torch operations in 32 bits, 64 where 32 lose what matters) and the
library's entry points.  Shapes follow the library: token-major matrices
[tokens x heads * head_dim], bf16, documents packed one behind the other with
their first rows in an int32 array of documents + 1 entries."""
from __future__ import annotations

import math
import random

import torch

own = False


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _norm(M, d, step, f32, bias):
    return {"op": "norm", "M": M, "d": d, "step": step, "f32": f32, "bias": bias}


def _tables(n_pos, rot, scaling, factor):
    return {"op": "tables", "n_pos": n_pos, "rot": rot, "scaling": scaling, "factor": factor}


def _rotary(M, heads, kv_heads, head_dim, rot, layout, inverse):
    return {"op": "rotary", "M": M, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "rot": rot,
            "layout": layout, "inverse": inverse, "n_pos": 8192}


def _attention(M, docs, lens, pad, heads, kv_heads, head_dim, step, causal=True, prefix=False, cap=0.0, bias=False):
    """M rows, the last `pad` of them behind the last document; `lens` 0: documents of one length, else the seed of
    their lengths."""
    return {"op": "attention", "M": M, "docs": docs, "lens": lens, "pad": pad, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "step": step, "causal": causal, "prefix": prefix, "cap": cap, "bias": bias}


def listed():
    named = [
        # the norm of one new token: latency alone
        ("norm, one token", _norm(1, 4096, False, False, True)),
        # the norm's training step in front of projections that are trained without a common gradient buffer
        ("norm step, 16384 tokens", _norm(16384, 4096, True, False, True)),
        # a wide norm without bias whose gradient comes as the fp32 sum that the projections' input gradients leave
        ("norm step, ragged fp32 gradient", _norm(1000, 14336, True, True, False)),
        # the tables of a context stretched to 131072 positions, built once when a model is loaded
        ("tables, 131072 positions", _tables(131072, 128, "wavelength", 8.0)),
        # q and k of a training batch, whole heads
        ("rotary, 16384 tokens", _rotary(16384, 32, 8, 128, 128, "half", False)),
        # the gradients of a partly rotated, interleaved layout at an odd number of tokens
        ("rotary back, ragged, part of a head", _rotary(3001, 20, 20, 80, 32, "interleaved", True)),
        # q and k of one new token
        ("rotary, one token", _rotary(1, 32, 8, 128, 128, "half", False)),
        # a short prompt: one tile of queries, latency alone
        ("attention, 96 tokens", _attention(96, 1, 0, 0, 32, 8, 128, False)),
        # the training step of a batch of four whole sequences
        ("attention step, 4 x 4096", _attention(16384, 4, 0, 0, 32, 8, 128, True)),
        # packed fine-tuning samples of many lengths with padding behind them; capped scores and a distance bias
        ("attention step, packed, cap and bias", _attention(8192, 23, 7, 131, 16, 16, 64, True, cap=30.0, bias=True)),
        # the prompt pass over one long document
        ("attention, one long document", _attention(16384, 1, 0, 0, 32, 8, 128, False)),
        # samples whose prompt sees itself both ways and whose answer is causal
        ("attention step, prefix", _attention(4000, 5, 3, 0, 32, 4, 128, True, prefix=True)),
    ]
    return [dict(c, name=n) for n, c in named]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm", "tables", "rotary", "rotary", "attention", "attention", "attention", "attention"])
    if kind == "norm":
        d = 8 * _log(rng, 8, 2048)
        M = max(1, min(_log(rng, 1, 20000), 16384 * 4096 // d))
        return _norm(M, d, rng.random() < 0.7, rng.random() < 0.4, rng.random() < 0.6)
    if kind == "tables":
        return _tables(_log(rng, 100, 131072), 16 * rng.randint(1, 8),
                       rng.choice(["none", "linear", "ntk", "wavelength", "ramp"]), rng.choice([2.0, 4.0, 8.0, 16.0]))
    if kind == "rotary":
        head_dim = 8 * rng.randint(2, 20)
        rot = 16 * rng.randint(1, head_dim // 16)
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4])
        M = max(1, min(_log(rng, 1, 40000), 16384 * 40 * 128 // ((heads + kv) * head_dim)))
        return _rotary(M, heads, kv, head_dim, rot, rng.choice(["half", "interleaved"]), rng.random() < 0.5)
    M = _log(rng, 1, 6000)
    docs = min(M, _log(rng, 1, 40))
    kv = rng.choice([1, 2, 4, 8])
    pad = 0 if rng.random() < 0.6 or M - docs < 2 else rng.randint(1, max(1, (M - docs) // 4))
    causal = rng.random() < 0.75
    return _attention(M, docs, rng.randint(1, 1 << 20), pad, kv * rng.choice([1, 2, 4]), kv, rng.choice([64, 128]),
                      rng.random() < 0.6, causal, causal and rng.random() < 0.3,
                      rng.choice([0.0, 0.0, 20.0, 50.0]), rng.random() < 0.3)


def _doc_starts(case):
    """First rows of the documents, and the end of the last one."""
    n, total = case["docs"], case["M"] - case["pad"]
    if not case["lens"]:
        return [total * i // n for i in range(n + 1)]
    r = random.Random(case["lens"])
    cuts = sorted(r.sample(range(1, total), n - 1)) if n > 1 else []
    return [0] + cuts + [total]


def _prefixes(case):
    """Rows at the head of each document that all of its rows see."""
    s = _doc_starts(case)
    lens = [b - a for a, b in zip(s, s[1:])]
    if not case["causal"]:
        return lens
    if not case["prefix"]:
        return [0] * len(lens)
    r = random.Random(case["lens"] + 1)
    return [r.randint(0, n) for n in lens]


def _pairs(case):
    """Visible (query, key) pairs of one head."""
    s, p = _doc_starts(case), _prefixes(case)
    return sum(n * (n + 1) // 2 + x * (x - 1) // 2 for n, x in ((b - a, x) for a, b, x in zip(s, s[1:], p)))


def work(case):
    if case["op"] == "norm":
        n = case["M"] * case["d"]
        vec = case["d"] * (4 if case["bias"] else 2)
        if not case["step"]:
            return {"bytes": 4 * n + vec + 8 * case["M"], "flops": 8 * n}
        # x once, dy once, y and dx once, mean and rstd, dg (and db)
        return {"bytes": (2 + (4 if case["f32"] else 2) + 2 + 2) * n + 3 * vec + 8 * case["M"], "flops": 20 * n}
    if case["op"] == "tables":
        return {"bytes": 4 * case["n_pos"] * case["rot"], "flops": 8 * case["n_pos"] * case["rot"]}
    if case["op"] == "rotary":
        n = case["M"] * (case["heads"] + case["kv_heads"])
        used = min(case["M"], case["n_pos"])
        return {"bytes": 4 * n * case["head_dim"] + 4 * used * case["rot"] + 4 * case["M"], "flops": 3 * n * case["rot"]}
    q, kv = case["M"] * case["heads"] * case["head_dim"], case["M"] * case["kv_heads"] * case["head_dim"]
    mul = 2 * _pairs(case) * case["heads"] * case["head_dim"]
    if not case["step"]:
        return {"bytes": 2 * (2 * q + 2 * kv) + 4 * case["M"] * case["heads"], "flops": 2 * mul}
    return {"bytes": 2 * (4 * q + 4 * kv) + 4 * case["M"] * case["heads"], "flops": 7 * mul}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _rotary_args(case):
    return {"base": 10000.0, "scaling": case.get("scaling", "none"), "factor": case.get("factor", 1.0),
            "low": 1.0, "high": 32.0 if case.get("scaling") == "ramp" else 4.0, "original": 8192,
            "amplitude": 1.2 if case.get("scaling") == "ramp" else 1.0}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "norm":
        M, d = case["M"], case["d"]
        # rows of different offsets and scales, as a residual stream has them
        s["X"] = (torch.randn(M, d, generator=gen, device="cuda") * (0.5 + torch.rand(M, 1, generator=gen, device="cuda"))
                  + 0.3 * torch.randn(M, 1, generator=gen, device="cuda")).to(torch.bfloat16)
        s["g"] = (0.5 + torch.rand(d, generator=gen, device="cuda")).to(torch.bfloat16)
        s["b"] = _normal(gen, d) if case["bias"] else None
        if case["step"]:
            dY = torch.randn(M, d, generator=gen, device="cuda")
            s["dY"] = dY if case["f32"] else dY.to(torch.bfloat16)
    elif case["op"] == "tables":
        # the base is the tables' only input value: each seed another
        s["base"] = 10000.0 + (seed % 1000003)
    elif case["op"] == "rotary":
        M, D = case["M"], case["head_dim"]
        s["Q"], s["K"] = _normal(gen, M, case["heads"] * D), _normal(gen, M, case["kv_heads"] * D)
        s["pos"] = torch.randint(0, case["n_pos"], (M,), generator=gen, device="cuda", dtype=torch.int32)
        ang = (torch.arange(case["n_pos"], device="cuda", dtype=torch.float64)[:, None]
               * 10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"]))
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
    else:
        M, D = case["M"], case["head_dim"]
        s["Q"], s["K"], s["V"] = (_normal(gen, M, h * D) for h in (case["heads"], case["kv_heads"], case["kv_heads"]))
        if case["step"]:
            s["dO"] = _normal(gen, M, case["heads"] * D)
        s["starts"] = torch.tensor(_doc_starts(case), dtype=torch.int32, device="cuda")
        s["prefix"] = torch.tensor(_prefixes(case), dtype=torch.int32, device="cuda") if case["prefix"] else None
        s["slopes"] = (torch.tensor([2.0 ** (-8.0 * (h + 1) / case["heads"]) for h in range(case["heads"])],
                                    device="cuda") if case["bias"] else None)
    if own:
        # what a program keeps from call to call: the workspace, and the plan
        # of a batch's documents, which all layers of a model share
        import lora_linear_fine_b200 as L
        if case["op"] == "attention":
            s["plan"] = L.AttentionPlan(s["starts"], case["M"], prefix_len=s["prefix"], causal=case["causal"])
            s["ws"] = L.Workspace(L.lora_linear_attn_workspace_size(L.make_attn_desc(
                case["M"], case["docs"], case["heads"], case["kv_heads"], case["head_dim"], case["causal"])))
        elif case["op"] == "norm":
            s["ws"] = L.Workspace(L.lora_linear_layernorm_workspace_size(case["M"], case["d"]))
        else:
            s["ws"] = L.Workspace(256)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else {"norm": _plain_norm, "tables": _plain_tables, "rotary": _plain_rotary,
                                    "attention": _plain_attention}[s["case"]["op"]](s)


def _run_own(s):
    import lora_linear_fine_b200 as L
    c = s["case"]
    if c["op"] == "norm":
        Y, mean, rstd = L.layer_norm(s["X"], s["g"], s["b"], 1e-5)
        out = {"Y": Y, "mean": mean, "rstd": rstd}
        if c["step"]:
            dX, dg, db = L.layer_norm_backward(s["dY"], s["X"], s["g"], mean, rstd, bias=c["bias"], workspace=s["ws"])
            out |= {"dX": dX, "dg": dg}
            if c["bias"]:
                out["db"] = db
        return out
    if c["op"] == "tables":
        cos, sin = L.rotary_tables(c["n_pos"], c["rot"], **(_rotary_args(c) | {"base": s["base"]}))
        return {"cos": cos, "sin": sin}
    if c["op"] == "rotary":
        Yq, Yk = L.rotary(s["Q"], s["K"], s["pos"], s["cos"], s["sin"], c["head_dim"], layout=c["layout"],
                          inverse=c["inverse"], workspace=s["ws"])
        return {"Q": Yq, "K": Yk}
    args = {"heads": c["heads"], "kv_heads": c["kv_heads"], "softcap": c["cap"], "slopes": s["slopes"]}
    O, lse = L.attention(s["Q"], s["K"], s["V"], s["plan"], **args)
    out = {"O": O, "lse": lse}
    if c["step"]:
        dQ, dK, dV = L.attention_backward(s["dO"], s["Q"], s["K"], s["V"], O, lse, s["plan"], workspace=s["ws"], **args)
        out |= {"dQ": dQ, "dK": dK, "dV": dV}
    return out


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_norm(s):
    c, x, g = s["case"], s["X"].float(), s["g"].float()
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1, keepdim=True) + 1e-5)
    xh = xc * rstd
    y = xh * g
    if c["bias"]:
        y = y + s["b"].float()
    out = {"Y": y.to(torch.bfloat16), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if c["step"]:
        dy = s["dY"].float()
        dh = dy * g
        dx = rstd * (dh - dh.mean(1, keepdim=True) - xh * (dh * xh).mean(1, keepdim=True))
        out |= {"dX": dx.to(torch.bfloat16), "dg": (dy * xh).sum(0)}
        if c["bias"]:
            out["db"] = dy.sum(0)
    return out


def _frequencies(base, rot, scaling, factor, low, high, original):
    """Angles per position (64 bits) of the rot / 2 pairs under a scaling for long contexts."""
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / factor
    elif scaling == "wavelength":   # by the turns that a pair makes over the original context
        keep = ((original * f / (2 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1 - keep)
    elif scaling == "ramp":         # by the pair's index between those of `high` and `low` turns
        at = [rot * math.log(original / (2 * math.pi * n)) / (2 * math.log(base)) for n in (high, low)]
        a, b = max(0.0, math.floor(at[0])), min(rot - 1.0, math.ceil(at[1]))
        keep = 1 - ((i - a) / max(b - a, 1e-3)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1 - keep)
    return f


def _plain_tables(s):
    c, a = s["case"], _rotary_args(s["case"])
    f = _frequencies(s["base"], c["rot"], a["scaling"], a["factor"], a["low"], a["high"], a["original"])
    ang = torch.arange(c["n_pos"], device="cuda", dtype=torch.float64)[:, None] * f
    return {"cos": (ang.cos() * a["amplitude"]).float(), "sin": (ang.sin() * a["amplitude"]).float()}


def _plain_rotary(s):
    c = s["case"]
    at = s["pos"].long()
    cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
    if c["inverse"]:
        sin = -sin

    def turned(x):
        x = x.float().view(c["M"], -1, c["head_dim"])
        r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        if c["layout"] == "half":
            a, b = r[..., :c["rot"] // 2], r[..., c["rot"] // 2:]
            r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        return torch.cat((r, rest), -1).reshape(c["M"], -1).to(torch.bfloat16)

    return {"Q": turned(s["Q"]), "K": turned(s["K"])}


def _plain_attention(s):
    """Document by document, as many heads at a time as keep the scores within 2^28 values."""
    c = s["case"]
    H, G, D, M = c["heads"], c["kv_heads"], c["head_dim"], c["M"]
    n, scale = H // G, 1.0 / math.sqrt(D)
    Q, K, V = s["Q"].view(M, G, n, D), s["K"].view(M, G, D), s["V"].view(M, G, D)
    O, lse = torch.zeros_like(s["Q"]), torch.full((M, H), -math.inf, device="cuda")
    out = {"O": O, "lse": lse}
    if c["step"]:
        dO = s["dO"].view(M, G, n, D)
        out |= {"dQ": torch.zeros_like(s["Q"]), "dK": torch.zeros_like(s["K"]), "dV": torch.zeros_like(s["V"])}
    starts = _doc_starts(c)
    for a, b, pre in zip(starts, starts[1:], _prefixes(c)):
        T = b - a
        i, j = torch.arange(T, device="cuda")[:, None], torch.arange(T, device="cuda")
        hidden = (j > i) & (j >= pre)
        few = max(1, min(G, (1 << 28) // (T * T * n)))
        for h in range(0, G, few):
            e = min(G, h + few)
            q = Q[a:b, h:e].float().permute(1, 2, 0, 3).reshape(e - h, n * T, D)
            k, v = (x[a:b, h:e].float().transpose(0, 1) for x in (K, V))
            z = (q @ k.transpose(1, 2)).view(e - h, n, T, T) * scale
            if c["cap"]:
                t = torch.tanh(z / c["cap"])
                z = c["cap"] * t
            if c["bias"]:
                z = z - s["slopes"].view(G, n, 1, 1)[h:e] * (i - j).abs()
            z = z.masked_fill(hidden, -math.inf)
            top = z.amax(-1, keepdim=True)
            p = torch.exp(z - top)
            tot = p.sum(-1, keepdim=True)
            p = p / tot
            lse.view(M, G, n)[a:b, h:e] = (top + torch.log(tot))[..., 0].permute(2, 0, 1)
            o = (p.view(e - h, n * T, T) @ v).view(e - h, n, T, D)
            O.view(M, G, n, D)[a:b, h:e] = o.permute(2, 0, 1, 3).to(torch.bfloat16)
            if c["step"]:
                do = dO[a:b, h:e].float().permute(1, 2, 0, 3).reshape(e - h, n * T, D)
                dp = (do @ v.transpose(1, 2)).view(e - h, n, T, T)
                dz = p * (dp - (p * dp).sum(-1, keepdim=True))
                if c["cap"]:
                    dz = dz * (1 - t * t)
                dz = (dz * scale).view(e - h, n * T, T)
                out["dQ"].view(M, G, n, D)[a:b, h:e] = (dz @ k).view(e - h, n, T, D).permute(2, 0, 1, 3).to(torch.bfloat16)
                out["dK"].view(M, G, D)[a:b, h:e] = (dz.transpose(1, 2) @ q).transpose(0, 1).to(torch.bfloat16)
                out["dV"].view(M, G, D)[a:b, h:e] = (p.view(e - h, n * T, T).transpose(1, 2) @ do).transpose(0, 1).to(torch.bfloat16)
    return out


# ---------------------------------------------------------------------------
# 64 bits: the definitions, with gradients by differentiation
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "tables": _exact_tables, "rotary": _exact_rotary,
            "attention": _exact_attention}[case["op"]](s)


def _exact_norm(s):
    c = s["case"]
    x, g = s["X"].double().requires_grad_(), s["g"].double().requires_grad_()
    b = s["b"].double().requires_grad_() if c["bias"] else None
    var, mean = torch.var_mean(x, 1, correction=0)
    rstd = (var + 1e-5).rsqrt()
    y = torch.einsum("md,m,d->md", x - mean[:, None], rstd, g)
    y = y if b is None else y + b
    out = {"Y": y.detach(), "mean": mean.detach(), "rstd": rstd.detach()}
    if c["step"]:
        got = torch.autograd.grad(y, [x, g] + ([b] if c["bias"] else []), s["dY"].double())
        out |= dict(zip(("dX", "dg", "db"), got))
    return out


def _exact_tables(s):
    c, a = s["case"], _rotary_args(s["case"])
    R, base, turns = c["rot"], s["base"], 2 * math.pi
    f = []
    for k in range(R // 2):
        w = math.exp(-2 * k / R * math.log(base))
        if c["scaling"] == "linear":
            w /= c["factor"]
        elif c["scaling"] == "ntk":
            if R > 2:
                w = math.exp(-2 * k / R * (math.log(base) + R / (R - 2) * math.log(c["factor"])))
        elif c["scaling"] == "wavelength":
            r = a["original"] * w / turns
            if r < a["low"]:
                w /= c["factor"]
            elif r <= a["high"]:
                m = (r - a["low"]) / (a["high"] - a["low"])
                w = (1 - m) * w / c["factor"] + m * w
        elif c["scaling"] == "ramp":
            lo = max(0, math.floor(R / 2 * math.log(a["original"] / (turns * a["high"]), base)))
            hi = min(R - 1, math.ceil(R / 2 * math.log(a["original"] / (turns * a["low"]), base)))
            m = 0.0 if k <= lo else 1.0 if k >= hi else (k - lo) / (hi - lo)
            w = m * w / c["factor"] + (1 - m) * w
        f.append(w)
    ang = torch.outer(torch.arange(c["n_pos"], dtype=torch.float64, device="cuda"),
                      torch.tensor(f, dtype=torch.float64, device="cuda"))
    z = torch.polar(torch.full_like(ang, a["amplitude"]), ang)
    return {"cos": z.real.contiguous(), "sin": z.imag.contiguous()}


def _exact_rotary(s):
    """Each pair as a complex number, turned by its unit factor."""
    c, R = s["case"], s["case"]["rot"]
    w = torch.complex(s["cos"].double(), s["sin"].double())[s["pos"].long()][:, None, :]
    w = w.conj() if c["inverse"] else w
    first = torch.arange(R // 2, device="cuda") * (1 if c["layout"] == "half" else 2)
    second = first + (R // 2 if c["layout"] == "half" else 1)

    def turned(x):
        y = x.double().view(c["M"], -1, c["head_dim"]).clone()
        z = torch.complex(y[..., first], y[..., second]) * w
        y[..., first], y[..., second] = z.real, z.imag
        return y.view(c["M"], -1)

    return {"Q": turned(s["Q"]), "K": turned(s["K"])}


def _exact_attention(s):
    c = s["case"]
    M, H, G, D = c["M"], c["heads"], c["kv_heads"], c["head_dim"]
    q, k, v = (s[n].double().view(M, -1, D) for n in "QKV")
    O, lse = torch.zeros_like(q), torch.full((M, H), -math.inf, dtype=torch.float64, device="cuda")
    grads = [torch.zeros_like(x) for x in (q, k, v)] if c["step"] else None
    starts = _doc_starts(c)
    for d, pre in enumerate(_prefixes(c)):
        rows = slice(starts[d], starts[d + 1])
        at = torch.arange(starts[d + 1] - starts[d], device="cuda", dtype=torch.float64)
        dist = at[:, None] - at[None, :]
        seen = (dist >= 0) | (at < pre)[None, :]
        for h in range(H):
            x = [t[rows, g].clone().requires_grad_(c["step"]) for t, g in ((q, h), (k, h * G // H), (v, h * G // H))]
            z = torch.einsum("id,jd->ij", x[0], x[1]) / D ** 0.5
            if c["cap"]:
                z = c["cap"] * torch.tanh(z / c["cap"])
            if c["bias"]:
                z = z - float(s["slopes"][h]) * dist.abs()
            z = torch.where(seen, z, torch.full_like(z, -math.inf))
            l = torch.logsumexp(z, 1)
            o = torch.exp(z - l[:, None]) @ x[2]
            O[rows, h], lse[rows, h] = o.detach(), l.detach()
            if c["step"]:
                for t, part, g in zip(grads, torch.autograd.grad(o, x, s["dO"].double().view(M, H, D)[rows, h]),
                                      (h, h * G // H, h * G // H)):
                    t[rows, g] += part
    out = {"O": O.view(M, -1), "lse": lse}
    if c["step"]:
        out |= {n: t.view(M, -1) for n, t in zip(("dQ", "dK", "dV"), grads)}
    return out
