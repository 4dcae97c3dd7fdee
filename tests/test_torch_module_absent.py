"""The torch functions without their short way into the library: they take the
long one, with a warning, and give the same bits."""
import pytest


@pytest.fixture(params=["absent", "of another torch"])
def without(request, tmp_path, monkeypatch):
    """The package with no module, or with one that cannot be loaded."""
    from lora_linear_fine_b200 import build
    build.build(quiet=True)
    import lora_linear_fine_b200 as L
    if request.param != "absent":
        (tmp_path / "_lora_torch.so").write_bytes(b"\x7fELF of another interpreter")
    monkeypatch.setattr(L, "_PKG", str(tmp_path))
    monkeypatch.setattr(L, "_torch", L._LazyTorch())
    return L


def test_calls_are_checked_as_ever(without):
    import torch
    L = without
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    with pytest.warns(RuntimeWarning, match="_lora_torch"), pytest.raises(L.LoraError, match="CUDA"):
        L.layer_norm(bf(4, 64), bf(64))
    with pytest.raises(L.LoraError, match="not contiguous"):
        L.layer_norm(bf(64, 4).t(), bf(64))


@pytest.mark.gpu
@pytest.mark.filterwarnings("ignore:.*_lora_torch")
def test_same_bits(without, monkeypatch):
    import torch
    L = without
    gen = torch.Generator().manual_seed(3)
    bf = lambda *s: torch.randn(*s, generator=gen).bfloat16().cuda()
    X, g, b, dY = bf(300, 256), bf(256), bf(256), bf(300, 256)
    V, dO = bf(300, 128), bf(300, 256)
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 130, 300], dtype=torch.int32, device="cuda")
    plan, ws = L.AttentionPlan(starts, 300), L.Workspace(1 << 24)

    def step():
        Y, mean, rstd = L.layer_norm(X, g, b)
        cos, sin = L.rotary_tables(300, 64, scaling="linear", factor=2.0)
        q, k = L.rotary(Y, Y[:, :128].contiguous(), pos, cos, sin, 64, workspace=ws)
        O, lse = L.attention(q, k, V, plan, 4, 2, softcap=20.0)
        return (Y, mean, rstd, cos, sin, q, k, O, lse, *L.layer_norm_backward(dY, X, g, mean, rstd, workspace=ws),
                *L.attention_backward(dO, q, k, V, O, lse, plan, 4, 2, softcap=20.0, workspace=ws))

    long = step()
    monkeypatch.undo()
    assert L._torch.layer_norm(X, g, b, 1e-5) is not None
    assert all(torch.equal(p, q) for p, q in zip(long, step()))
