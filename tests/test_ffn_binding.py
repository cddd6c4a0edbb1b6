"""The binding's own helpers, without a GPU."""
import torch

import gemv_w4a16_w8a8_b200 as qg


class Stream:
    cuda_stream = 1234


def test_device_and_stream_by_torchs_public_names(monkeypatch):
    """torch's private shortcuts to the current device and stream may go; its public names stay."""
    monkeypatch.delattr(torch._C, "_cuda_getDevice", raising=False)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: (index, Stream())[1])

    class Tensor:
        def get_device(self):
            return 3

    assert qg._elsewhere(Tensor(), None) is False and qg._elsewhere(Tensor(), 7) is True
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert qg._elsewhere(Tensor(), None) is True
    assert qg._current(3) == 1234
