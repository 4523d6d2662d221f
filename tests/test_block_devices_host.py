"""The feed-forward block's tensors on more than one device, or on one that is not the
current one: refused or entered before an address reaches a kernel.  Stand-ins for
tensors and for the library's calls; nothing touches a GPU."""
import torch

from .test_devices_host import Tensor, lib  # noqa: F401
import pytest

B = torch.bfloat16


def _tensors(op, dev=0, **other):
    shapes = {"x": (4, 16), "wg": (40, 16), "wu": (40, 16), "wd": (16, 40), "residual": (4, 16), "y": (4, 16), "dy": (4, 16)}
    t = {k: Tensor(s, B, other.get(k, dev)) for k, s in shapes.items()}
    t["saved"] = Tensor(op._saved.shape, torch.uint8, other.get("saved", dev))
    t["workspace"] = Tensor((1 << 24,), torch.uint8, other.get("workspace", dev))
    return t


@pytest.fixture
def block(lib, monkeypatch):  # noqa: F811
    for f in ("gated_ffn_fwd", "gated_ffn_bwd"):
        monkeypatch.setattr(lib.head.head_capi, f, lambda *a, f=f: lib.calls.append((f, lib.current, a[-1])))
    lib.op = lib.head.GatedFeedForward(4, 16, 40, "bf16")
    return lib


FORWARD, BACKWARD = ("x", "wg", "wu", "wd", "residual", "y", "workspace"), ("dy", "x", "wg", "wu", "wd", "saved", "workspace")


@pytest.mark.parametrize("names,call", [(FORWARD, "__call__"), (BACKWARD, "backward")])
def test_tensors_of_another_device_are_refused(block, names, call):
    for odd in names:
        for dev in (1, -1):
            t = _tensors(block.op, **{odd: dev})
            with pytest.raises(ValueError):
                getattr(block.op, call)(**{k: t[k] for k in names})
    assert not block.calls


@pytest.mark.parametrize("names,call,f", [(FORWARD, "__call__", "gated_ffn_fwd"), (BACKWARD, "backward", "gated_ffn_bwd")])
def test_a_call_runs_on_its_tensors_device(block, names, call, f):
    t = _tensors(block.op, dev=1)
    getattr(block.op, call)(**{k: t[k] for k in names})
    assert block.calls == [(f, 1, 101)] and block.current == 0
