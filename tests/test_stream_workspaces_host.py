"""Which default workspaces a device report costs: those whose counters a wait that
ran out may have left, on the device that reported it, and no others."""
import types

import pytest
import torch

from speculative_decode_verify_w4a16_gb300 import _lib, api

KEYS = [(0, 11, "kv16_attention", False), (0, 12, "kv16_attention", True), (0, 11, "kv8_tree_attention", False),
        (1, 13, "kv16_attention", False)]


@pytest.mark.parametrize("status,kept", [
    (_lib.OK, KEYS), (_lib.ERR_DEVICE_INPUT, KEYS), (_lib.ERR_BOUNDS, KEYS), (_lib.ERR_CUDA, KEYS),
    (_lib.ERR_DEVICE_TIMEOUT, KEYS[2:]),
])
def test_what_a_report_drops(monkeypatch, status, kept):
    held = {k: (0, object()) for k in KEYS}
    monkeypatch.setattr(api, "_stream_ws", dict(held))
    monkeypatch.setattr(api, "_device", lambda: 0)
    monkeypatch.setattr(api, "lib", lambda: types.SimpleNamespace(w4a16_check_device_status=lambda stream: status))
    assert api.check_device_status(types.SimpleNamespace(cuda_stream=11)) == status
    assert list(api._stream_ws) == kept and all(api._stream_ws[k] is held[k] for k in kept)


def test_workspaces_of_one_s_own():
    """An expanded tensor counts more elements than it has bytes: refused before a kernel writes past it."""
    def ws(t, device=0):
        return types.SimpleNamespace(get_device=lambda: device, device=f"cuda:{device}", is_contiguous=t.is_contiguous)
    api._need_ws(ws(torch.zeros(64, dtype=torch.uint8)), 0)
    for bad in (ws(torch.zeros(1, dtype=torch.uint8).expand(1 << 20)), ws(torch.zeros(64)[::2]), ws(torch.zeros(64), 1)):
        with pytest.raises(ValueError):
            api._need_ws(bad, 0)
