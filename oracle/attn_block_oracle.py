"""fp64 statements (numpy) of the operators around the attention of a packed
batch: layer norm, rotary positions, attention over documents, each with its
gradient.  Plain loops over documents and heads; no blocking, no library
attention."""
from __future__ import annotations

import numpy as np


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
def layer_norm(X, g, b, eps):
    """(Y, mean, rstd)."""
    mean = X.mean(axis=1)
    rstd = 1.0 / np.sqrt(((X - mean[:, None]) ** 2).mean(axis=1) + eps)
    Y = (X - mean[:, None]) * rstd[:, None] * g
    return (Y if b is None else Y + b), mean, rstd


def layer_norm_backward(dY, X, g, eps):
    """(dX, dg, db)."""
    _, mean, rstd = layer_norm(X, g, None, eps)
    xh = (X - mean[:, None]) * rstd[:, None]
    dh = dY * g
    dX = rstd[:, None] * (dh - dh.mean(axis=1)[:, None] - xh * (dh * xh).mean(axis=1)[:, None])
    return dX, (dY * xh).sum(axis=0), dY.sum(axis=0)


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def rotary_frequencies(rot, base=10000.0, scaling="none", factor=1.0, low=1.0, high=4.0, original=8192):
    """Angle per position of each of the rot / 2 pairs."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2.0))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor
    if scaling == "wavelength":
        keep = np.clip((original * f / (2 * np.pi) - low) / (high - low), 0.0, 1.0)
    elif scaling == "ramp":
        at = lambda turns: rot * np.log(original / (2 * np.pi * turns)) / (2 * np.log(base))
        first, last = max(0.0, np.floor(at(high))), min(rot - 1.0, np.ceil(at(low)))
        keep = 1.0 - np.clip((i - first) / max(last - first, 1e-3), 0.0, 1.0)
    else:
        return f
    return f * keep + f / factor * (1.0 - keep)


def rotary_tables(n_pos, rot, amplitude=1.0, **kw):
    ang = np.arange(n_pos, dtype=np.float64)[:, None] * rotary_frequencies(rot, **kw)
    return np.cos(ang) * amplitude, np.sin(ang) * amplitude


def rotary(X, pos, cos, sin, head_dim, layout="half", inverse=False):
    """X [M x heads * head_dim] turned at the table rows pos."""
    M, rot = X.shape[0], 2 * cos.shape[1]
    y = X.reshape(M, -1, head_dim).copy()
    c, s = cos[pos][:, None, :], (-sin if inverse else sin)[pos][:, None, :]
    ia = np.arange(rot // 2) if layout == "half" else np.arange(0, rot, 2)
    ib = ia + (rot // 2 if layout == "half" else 1)
    a, b = X.reshape(M, -1, head_dim)[:, :, ia], X.reshape(M, -1, head_dim)[:, :, ib]
    y[:, :, ia], y[:, :, ib] = a * c - b * s, b * c + a * s
    return y.reshape(M, -1)


# ---------------------------------------------------------------------------
# attention over packed documents
# ---------------------------------------------------------------------------
def visible(n, prefix, causal):
    """[n x n]: whether row i of a document sees key j."""
    i, j = np.arange(n)[:, None], np.arange(n)[None, :]
    return (j <= i) | (j < prefix) if causal else np.ones((n, n), dtype=bool)


def attention(Q, K, V, starts, heads, kv_heads, prefix=None, causal=True, scale=None, softcap=0.0, slopes=None,
              dO=None, bounds=False, fp=2.0 ** -14):
    """Forward, and with dO the gradients: a dict of O, lse (dQ, dK, dV).

    bounds: also, under "tol", how far each output of a kernel may be off that
    rounds p and ds to bf16 for their products (half a step, 2^-8 relative,
    each), its outputs to bf16, and computes everything else in fp32 to a
    relative `fp` of the terms it adds: 2^-14 for scores of magnitude up to 2^3
    (fp32 products of up to 2^7 features or sums of up to 2^9 keys lose at most
    2^9 half steps of 2^-24 each, and a score of magnitude up to 2^3 turns its
    own error into a relative error of p eight times as large)."""
    M = Q.shape[0]
    D = Q.shape[1] // heads
    scale = D ** -0.5 if scale is None else scale
    q, k, v = (x.reshape(M, -1, D) for x in (Q, K, V))
    out = {"O": np.zeros((M, heads, D)), "lse": np.full((M, heads), -np.inf)}
    tol = {"O": np.zeros((M, heads, D)), "lse": np.zeros((M, heads))}
    if dO is not None:
        g = dO.reshape(M, heads, D)
        for name, like in (("dQ", q), ("dK", k), ("dV", v)):
            out[name], tol[name] = np.zeros_like(like), np.zeros_like(like)
    half = 2.0 ** -8
    for d in range(len(starts) - 1):
        a, e = int(starts[d]), int(starts[d + 1])
        n = e - a
        if n == 0:
            continue
        see = visible(n, 0 if prefix is None else int(prefix[d]), causal)
        dist = np.abs(np.arange(n)[:, None] - np.arange(n)[None, :])
        for h in range(heads):
            c = h * kv_heads // heads
            qh, kh, vh = q[a:e, h], k[a:e, c], v[a:e, c]
            z = scale * (qh @ kh.T)
            t = np.zeros_like(z)
            if softcap > 0:
                t = np.tanh(z / softcap)
                z = softcap * t
            if slopes is not None:
                z = z - slopes[h] * dist
            z = np.where(see, z, -np.inf)
            top = z.max(axis=1, keepdims=True)
            p = np.exp(z - top)
            tot = p.sum(axis=1, keepdims=True)
            p /= tot
            o = p @ vh
            out["O"][a:e, h], out["lse"][a:e, h] = o, (top + np.log(tot))[:, 0]
            if bounds:
                tol["O"][a:e, h] = (half + fp) * (p @ np.abs(vh)) + half * np.abs(o)
                tol["lse"][a:e, h] = fp * (1 + np.abs(top[:, 0]))
            if dO is None:
                continue
            gh = g[a:e, h]
            dp = gh @ vh.T
            delta = (gh * o).sum(axis=1, keepdims=True)
            ds = scale * p * (dp - delta) * (1 - t * t)
            out["dQ"][a:e, h] = ds @ kh
            out["dK"][a:e, c] += ds.T @ qh
            out["dV"][a:e, c] += p.T @ gh
            if bounds:
                off = (np.abs(gh) * tol["O"][a:e, h]).sum(axis=1, keepdims=True)      # of delta, from the rounded O
                size = np.abs(gh) @ np.abs(vh).T + (np.abs(gh) * (p @ np.abs(vh))).sum(axis=1, keepdims=True)
                ds_off = half * np.abs(ds) + (1 + half) * scale * p * (off + fp * size)
                tol["dQ"][a:e, h] = ds_off @ np.abs(kh) + half * np.abs(out["dQ"][a:e, h])
                tol["dK"][a:e, c] += ds_off.T @ np.abs(qh)
                tol["dV"][a:e, c] += (half + fp) * (p.T @ np.abs(gh))
    if dO is not None and bounds:
        for name in ("dK", "dV"):
            tol[name] += half * np.abs(out[name])
    res = {name: (x if name == "lse" else x.reshape(M, -1)) for name, x in out.items()}
    if bounds:
        res["tol"] = {name: (x if name == "lse" else x.reshape(M, -1)) for name, x in tol.items()}
    return res
