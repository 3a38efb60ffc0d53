"""The operators' binding (no GPU needed)."""
import pytest
import torch

lib = pytest.importorskip("lora_expert_gemm_amd")


class Current:
    cuda_stream = 0x70


@pytest.mark.parametrize("raw", [True, False])
def test_current_stream_with_and_without_torchs_raw_getter(monkeypatch, raw):
    """The raw getter is torch's own and not part of its interface: without
    it the current stream comes from the public call."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Current)
    if raw:
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0x70 + dev, raising=False)
    else:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert lib._where(None) == (0x70, 0)
