"""A plan's status is read on the plan's device, whichever is the current one."""
from types import SimpleNamespace

import pytest


@pytest.mark.parametrize("current", [0, 1])
def test_status_is_read_on_the_plans_device(monkeypatch, current):
    import lora_linear_fine_b200 as L
    import torch
    state = {"device": current}

    class On:
        def __init__(self, device):
            self.device = torch.device(device)

        def __enter__(self):
            self.before, state["device"] = state["device"], self.device.index

        def __exit__(self, *exc):
            state["device"] = self.before

    seen = []
    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: SimpleNamespace(cuda_stream=100 + state["device"]))
    monkeypatch.setattr(L, "lora_linear_device_status",
                        lambda ptr, stream: (seen.append((ptr, stream, state["device"])), (7, 2))[1])
    plan = object.__new__(L.AttentionPlan)
    plan.buf = SimpleNamespace(device=torch.device("cuda", 1), data_ptr=lambda: 4096)
    assert plan.status() == 2
    assert seen == [(4096, 101, 1)] and state["device"] == current
    assert plan.status(SimpleNamespace(cuda_stream=7)) == 2 and seen[1] == (4096, 7, 1)
