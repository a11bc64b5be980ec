"""The stream a call of the binding is enqueued on: torch's current stream of the
current device, asked for by its raw handle, or the one that is given."""
import pytest
import torch

from error_compensated_bit_echo_amd import binding as B


def test_current_device_is_asked(monkeypatch):
    """a current device other than the first, without needing one"""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 5)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x1000 + device)
    assert B._stream(None) == 0x1005


def test_given_streams_are_taken():
    class Stream:
        cuda_stream = 0x77

    assert B._stream(Stream()) == 0x77 and B._stream(0x88) == 0x88 and B._stream(0) == 0


@pytest.mark.gpu
def test_raw_handle_is_the_current_streams():
    assert B._stream(None) == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert B._stream(None) == side.cuda_stream == torch.cuda.current_stream().cuda_stream
        for device in range(torch.cuda.device_count()):  # every device there is
            with torch.cuda.device(device):
                assert B._stream(None) == torch.cuda.current_stream(device).cuda_stream
    assert B._stream(None) == torch.cuda.current_stream().cuda_stream
