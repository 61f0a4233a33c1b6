"""What dg_adamw_step checks of its arguments against the plan."""
import types

import pytest
import torch

import grouped_fp8_weight_gb300 as dg
from grouped_fp8_weight_gb300 import binding as B


def scalar(device):
    """Stands in for a scalar on a device that this machine may not have."""
    return types.SimpleNamespace(dtype=torch.float32, numel=lambda: 1, is_cuda=True,
                                 device=torch.device(device), data_ptr=lambda: 0x10000)


def plan(monkeypatch, device):
    """A plan on a device, and what its step hands to the library."""
    calls = []
    monkeypatch.setattr(B, "lib", lambda: types.SimpleNamespace(
        dg_adamw_step=lambda *a: calls.append(a) or B.DG_OK))
    monkeypatch.setattr(B, "_stream", lambda stream, t=None: 0)
    return B.AdamwPlan([[None]], None, B.DG_F32, 32, torch.device(device)), calls


@pytest.mark.parametrize("theirs", ["cuda:1", "cuda:2"])
def test_a_scale_on_another_device_is_refused(monkeypatch, theirs):
    p, calls = plan(monkeypatch, "cuda:0")
    with pytest.raises(ValueError, match="cuda:0"):
        dg.dg_adamw_step(p, 1, 1e-3, grad_scale=scalar(theirs))
    assert not calls


def test_a_scale_on_the_plan_s_device_is_passed_on(monkeypatch):
    p, calls = plan(monkeypatch, "cuda:1")
    dg.dg_adamw_step(p, 1, 1e-3, grad_scale=scalar("cuda:1"))
    dg.dg_adamw_step(p, 2, 1e-3)
    assert len(calls) == 2 and 0x10000 in calls[0] and 0x10000 not in calls[1]
