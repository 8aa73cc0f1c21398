"""Host-side behaviour of the block operators' Python binding (no GPU)."""

import types

import pytest

from bit_weight_only_awq_gb300 import build as awq_build

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def awq():
    awq_build.build()
    from bit_weight_only_awq_gb300 import awq as mod
    return mod


def test_workspace_sizes_are_a_devices_own(awq, monkeypatch):
    """The size follows the device's number of SMs: one remembered for a device is not another's, nor the caller's."""
    sms = [152]
    monkeypatch.setattr(awq, "lib", types.SimpleNamespace(kv4_attention_workspace_bytes=lambda *shape: 1000 * sms[0]))
    shape = (3, 3, 1, 12, 4, 64)
    assert awq.kv4_attention_workspace_bytes(*shape) == 152000
    assert awq._kv4_workspace_need(90, *shape) == 152000
    sms[0] = 16
    assert awq.kv4_attention_workspace_bytes(*shape) == 16000
    assert awq._kv4_workspace_need(91, *shape) == 16000 and awq._kv4_workspace_need(90, *shape) == 152000


def test_tensors_of_another_device_are_refused(awq, monkeypatch):
    def on(device):
        return types.SimpleNamespace(get_device=lambda: device)

    monkeypatch.setattr(awq, "_current_device", lambda: 1)
    awq._on_current_gpu("op", on(1), None, on(1))
    for tensors in ((on(0),), (on(1), on(0)), (on(1), None, on(-1))):
        with pytest.raises(ValueError, match="op: every tensor is on the current GPU"):
            awq._on_current_gpu("op", *tensors)
