"""Host side of the small calls (CPU)."""
import torch

from nvfp4_block_quantization_amax_b200 import api


def test_current_device_without_torchs_short_way(monkeypatch):
    """A torch without _cuda_getDevice is asked the long way; a call for the
    current device is made, not handed on to itself without end."""
    monkeypatch.setattr(api, "_current_device", None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert not api._elsewhere(torch.device("cuda", 1)) and api._elsewhere(torch.device("cuda", 0))
    monkeypatch.setattr(api, "_current_device", lambda: 0)
    assert api._elsewhere(torch.device("cuda", 1)) and not api._elsewhere(torch.device("cuda", 0))
