"""Workspaces of calls on a stream of the caller's."""
import pytest

pytestmark = pytest.mark.gpu


def _calls():
    import lora_linear_fine_b200 as L
    import torch
    bf = lambda *s: torch.randn(*s, device="cuda").bfloat16()
    X, g, dY = bf(64, 512), bf(512), bf(64, 512)
    _, mean, rstd = L.layer_norm(X, g)
    yield "layer_norm_backward", 1 << 20, lambda ws, st: L.layer_norm_backward(dY, X, g, mean, rstd, workspace=ws, stream=st)
    Q, K = bf(64, 256), bf(64, 128)
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    cos, sin = L.rotary_tables(64, 64)
    yield "rotary", 1 << 20, lambda ws, st: L.rotary(Q, K, pos, cos, sin, 64, workspace=ws, stream=st)
    V, dO = bf(64, 128), bf(64, 256)
    plan = L.AttentionPlan(torch.tensor([0, 64], dtype=torch.int32, device="cuda"), 64)
    O, lse = L.attention(Q, K, V, plan, 4, 2)
    yield "attention_backward", 1 << 20, lambda ws, st: L.attention_backward(dO, Q, K, V, O, lse, plan, 4, 2, workspace=ws,
                                                                             stream=st)


def test_a_workspace_outlives_the_work_on_another_stream():
    """A workspace that its owner drops while a stream still works in it is not
    handed out again before that stream is through."""
    import lora_linear_fine_b200 as L
    import torch
    for name, nbytes, call in _calls():
        call(L.Workspace(nbytes), None)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        ws = L.Workspace(nbytes)
        torch.cuda.synchronize()
        at = ws.buf.data_ptr()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)          # some fifty milliseconds
        call(ws, side)
        del ws
        again = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        assert not side.query(), "the stream was done too early to tell"
        assert again.data_ptr() != at, name
        side.synchronize()
