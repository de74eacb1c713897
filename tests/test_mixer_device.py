"""The token-mixer calls run on the device of their operands, whichever is current: with a library, a device and streams
that are stand-ins (no GPU needed)."""
import types

import pytest
import torch

from gated_delta_rule_29_gb300 import binding as B
from gated_delta_rule_29_gb300 import mixer


@pytest.fixture
def two_devices(monkeypatch):
    """Two devices, the first one current, and a library call that notes the current one and its stream."""
    now, calls = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *_):
            now[0] = self.before

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(mixer, "_current_device", lambda: now[0], raising=False)
    monkeypatch.setattr(mixer, "_raw_stream", lambda device: 100 + device)
    monkeypatch.setitem(mixer._functions, "glr_fwd", lambda p, stream: calls.append((now[0], stream)) or 0)
    return now, calls


@pytest.mark.parametrize("device", [0, 1])
def test_the_operands_device_is_current_during_the_call(two_devices, device):
    now, calls = two_devices
    mixer._call("glr_fwd", B.GlrFwdParams(), types.SimpleNamespace(get_device=lambda: device))
    assert calls == [(device, 100 + device)] and now == [0]


def test_the_device_is_put_back_after_an_error(two_devices, monkeypatch):
    now, _ = two_devices
    monkeypatch.setitem(mixer._functions, "glr_fwd", lambda p, stream: B.LA_ERR_INVALID_ARG)
    with pytest.raises(B.LinAttnError):
        mixer._call("glr_fwd", B.GlrFwdParams(), types.SimpleNamespace(get_device=lambda: 1))
    assert now == [0]


class CudaOperand(torch.Tensor):
    """A CPU tensor that says it is on cuda:0."""
    is_cuda = True
    device = torch.device("cuda", 0)


def test_a_stream_of_another_device_is_refused():
    x = torch.zeros(4, 8).as_subclass(CudaOperand)
    calls = mixer._on_stream(lambda x, stream=None: "ran")
    assert calls(x) == "ran"
    with pytest.raises(ValueError, match="stream must be on cuda:0"):
        calls(x, stream=types.SimpleNamespace(device=torch.device("cuda", 1)))
    with pytest.raises(ValueError, match="stream must be on cuda:0"):
        calls(x=x, stream=types.SimpleNamespace(device=torch.device("cuda", 1)))
