"""Argument checks of layer norm, rotary positions and attention: every bad
argument is answered on the host before a launch (and, through the torch
functions, as a LoraError)."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from lora_linear_fine_b200 import build
    build.build(quiet=True)
    import lora_linear_fine_b200 as L
    return L


def test_layernorm(lib):
    f = lambda X=16, g=16, b=16, M=4, d=64, eps=1e-5, Y=16, mean=16, rstd=16: lib.lora_linear_layernorm_fwd(
        X, g, b, M, d, eps, Y, mean, rstd, None)
    assert f(X=None) == 1 and f(g=None) == 1 and f(Y=None) == 1 and f(mean=None) == 1 and f(rstd=None) == 1
    assert f(M=-1) == 1 and f(d=0) == 1 and f(eps=-1.0) == 1 and f(eps=float("nan")) == 1
    assert f(d=60) == 2 and f(X=24) == 2 and f(g=24) == 2 and f(b=24) == 2 and f(Y=24) == 2 and f(mean=18) == 2
    assert f(d=16392) == 3
    assert f(b=None) not in (1, 2, 3)               # the shift is optional
    assert f(M=0, X=None, Y=None, mean=None, rstd=None) not in (1, 2, 3)
    assert lib.lora_linear_layernorm_workspace_size(100, 60) == 0
    assert lib.lora_linear_layernorm_workspace_size(100, 16392) == 0
    assert lib.lora_linear_layernorm_workspace_size(-1, 64) == 0
    assert lib.lora_linear_layernorm_workspace_size(0, 64) >= 256
    n = lib.lora_linear_layernorm_workspace_size(4, 64)
    b = lambda dY=16, f32=0, X=16, g=16, mean=16, rstd=16, M=4, d=64, dX=16, dg=16, db=16, ws=16, nb=n: \
        lib.lora_linear_layernorm_bwd(dY, f32, X, g, mean, rstd, M, d, dX, dg, db, ws, nb, None)
    assert b(dY=None) == 1 and b(X=None) == 1 and b(dX=None) == 1 and b(mean=None) == 1 and b(f32=2) == 1
    assert b(dY=24) == 2 and b(dX=24) == 2 and b(dg=18) == 2 and b(db=18) == 2
    assert b(ws=None) == 5 and b(nb=n - 1) == 5 and b(ws=24) == 5
    assert b(d=16392, nb=1 << 40) == 3


def test_rotary_tables(lib):
    def f(n_pos=8, rot=64, cos=16, sin=16, **kw):
        return lib.lora_linear_rotary_tables(lib.make_rotary_table_desc(n_pos, rot, **kw), cos, sin, None)
    assert f(n_pos=-1) == 1 and f(base=1.0) == 1 and f(base=float("inf")) == 1 and f(amplitude=0.0) == 1
    assert f(scaling="linear", factor=0.5) == 1 and f(scaling=5) == 1 and f(cos=None) == 1 and f(sin=None) == 1
    assert f(scaling="wavelength", factor=2.0, low=4.0, high=4.0) == 1
    assert f(scaling="ramp", factor=2.0, low=0.0) == 1 and f(scaling="ramp", factor=2.0, original=0) == 1
    assert f(rot=24) == 3 and f(rot=0) == 3 and f(rot=272) == 3
    assert f(cos=24) == 2 and f(sin=24) == 2


def test_rotary(lib):
    def f(M=4, heads=2, kv=1, hd=64, rot=32, layout="half", inverse=0, pos=16, cos=16, sin=16, n_pos=8, Q=16, K=32,
          Yq=48, Yk=64, ws=16, nb=256):
        return lib.lora_linear_rotary(lib.make_rotary_desc(M, heads, kv, hd, rot, layout, inverse),
                                      lib.make_rope_desc(pos, cos, sin, n_pos, hd), Q, K, Yq, Yk, ws, nb, None)
    assert f(M=-1) == 1 and f(heads=0) == 1 and f(kv=-1) == 1 and f(layout=2) == 1 and f(inverse=2) == 1
    assert f(Q=None) == 1 and f(K=None) == 1 and f(Yq=None) == 1 and f(Yk=None) == 1 and f(pos=None) == 1
    assert f(n_pos=0) == 1 and f(cos=None) == 1
    assert f(Yq=16) == 1 and f(Yk=32) == 1               # one in place, the other not
    assert f(hd=60) == 3 and f(hd=264, rot=32) == 3 and f(rot=24) == 3 and f(rot=80) == 3 and f(rot=0) == 3
    assert f(Q=24) == 2 and f(Yk=72) == 2 and f(cos=24) == 2 and f(pos=18) == 2
    assert f(ws=None) == 5 and f(nb=255) == 5
    assert f(kv=0, K=None, Yk=None) not in (1, 2, 3, 5)
    assert f(Yq=16, Yk=32) not in (1, 2, 3, 5)           # both in place


def test_attention_plan(lib):
    n = lib.lora_linear_attn_plan_size(1000, 3)
    assert n > 256
    assert lib.lora_linear_attn_plan_size(-1, 3) == 0 and lib.lora_linear_attn_plan_size(10, -1) == 0
    assert lib.lora_linear_attn_plan_size((1 << 30) + 1, 1) == 0
    assert lib.lora_linear_attn_plan_size(0, 0) >= 256
    f = lambda starts=16, pre=None, M=1000, docs=3, causal=1, plan=16, nb=n: lib.lora_linear_attn_plan(
        starts, pre, M, docs, causal, plan, nb, None)
    assert f(starts=None) == 1 and f(M=-1) == 1 and f(docs=-1) == 1 and f(causal=2) == 1
    assert f(starts=18) == 2 and f(pre=18) == 2
    assert f(M=(1 << 30) + 1) == 3
    assert f(plan=None) == 5 and f(plan=24) == 5 and f(nb=n - 1) == 5


def test_attention(lib):
    mk = lambda M=64, docs=1, h=4, g=2, D=64, **kw: lib.make_attn_desc(M, docs, h, g, D, **kw)
    n = lib.lora_linear_attn_plan_size(64, 1)

    def f(desc=None, plan=16, nb=n, Q=16, K=16, V=16, slopes=None, O=16, lse=16):
        return lib.lora_linear_attn_fwd(desc or mk(), plan, nb, Q, K, V, slopes, O, lse, None)
    assert f(mk(M=-1)) == 1 and f(mk(h=3)) == 1 and f(mk(g=0)) == 1 and f(mk(docs=-1)) == 1 and f(mk(causal=2)) == 1
    assert f(mk(scale=0.0)) == 1 and f(mk(scale=float("inf"))) == 1 and f(mk(softcap=-1.0)) == 1
    assert f(mk(softcap=float("nan"))) == 1 and f(mk(scale=-1.0)) == 1
    assert f(mk(D=80)) == 3 and f(mk(D=256)) == 3 and f(mk(h=8192, g=2)) == 3
    assert f(Q=None) == 1 and f(K=None) == 1 and f(V=None) == 1 and f(O=None) == 1 and f(lse=None) == 1
    assert f(Q=24) == 2 and f(O=24) == 2 and f(lse=18) == 2 and f(slopes=18) == 2
    assert f(plan=None) == 5 and f(nb=n - 1) == 5 and f(plan=24) == 5
    w = lib.lora_linear_attn_workspace_size(mk())
    assert w >= 256 + 64 * 4 * 4 and lib.lora_linear_attn_workspace_size(mk(D=80)) == 0

    def b(desc=None, plan=16, nb=n, dO=16, Q=16, K=16, V=16, O=16, lse=16, slopes=None, dQ=16, dK=16, dV=16, ws=16,
          wb=w):
        return lib.lora_linear_attn_bwd(desc or mk(), plan, nb, dO, Q, K, V, O, lse, slopes, dQ, dK, dV, ws, wb, None)
    for name in ("dO", "Q", "K", "V", "O", "lse", "dQ", "dK", "dV"):
        assert b(**{name: None}) == 1, name
        assert b(**{name: 18 if name == "lse" else 24}) == 2, name
    assert b(ws=None) == 5 and b(wb=w - 1) == 5 and b(plan=None) == 5


def test_torch_functions_refuse(lib):
    """Wrong types, shapes and devices never reach the library."""
    import torch
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    f32 = torch.zeros
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    bad = [
        lambda: lib.layer_norm(bf(4, 64), bf(64)),                                     # not on a GPU
        lambda: lib.layer_norm(f32(4, 64), bf(64)),
        lambda: lib.layer_norm(bf(4, 64), bf(32)),
        lambda: lib.layer_norm(bf(64, 4).t(), bf(64)),
        lambda: lib.layer_norm_backward(bf(4, 64).half(), bf(4, 64), bf(64), f32(4), f32(4)),
        lambda: lib.rotary_tables(8, 32, scaling="cubic"),
        lambda: lib.rotary_tables(8, 32, device="cpu"),
        lambda: lib.rotary(bf(4, 128), None, i32(4), f32(8, 16), f32(8, 16), 64),      # not on a GPU
        lambda: lib.rotary(bf(4, 100), None, i32(4), f32(8, 16), f32(8, 16), 64),
        lambda: lib.rotary(bf(4, 128), None, i32(3), f32(8, 16), f32(8, 16), 64),
        lambda: lib.rotary(bf(4, 128), None, i32(4).long(), f32(8, 16), f32(8, 16), 64),
        lambda: lib.rotary(bf(4, 128), None, i32(4), f32(8, 16), f32(8, 16), 64, layout="other"),
        lambda: lib.AttentionPlan(i32(3), 64),                                         # not on a GPU
        lambda: lib.AttentionPlan(i32(3).long(), 64),
        lambda: lib.AttentionPlan(i32(3), -1),
    ]
    for k, call in enumerate(bad):
        with pytest.raises(lib.LoraError):
            call()
            pytest.fail(f"call {k} was not refused")
