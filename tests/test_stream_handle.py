"""The stream that the row operators launch on: torch's current one, by its raw
handle, or by the Stream object where torch does not give the handle."""
import types

import pytest
import torch

import thread_register_tile_amd as trt


def launched_on(dev):
    seen = []
    trt._on(dev, lambda s: seen.append(s) or trt.OK)
    return seen


def test_without_the_raw_handle(monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for handle, want in ((0x77, 0x77), (0, None)):
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device: types.SimpleNamespace(cuda_stream=handle))
        assert launched_on(torch.device("cuda", 0)) == [want]


@pytest.mark.gpu
def test_both_name_the_same_stream(monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev, side = torch.device("cuda", torch.cuda.current_device()), torch.cuda.Stream()
    for st in (side, torch.cuda.current_stream()):
        with torch.cuda.stream(st):
            assert launched_on(dev) == [st.cuda_stream or None]
            with monkeypatch.context() as m:
                m.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
                assert launched_on(dev) == [st.cuda_stream or None]
