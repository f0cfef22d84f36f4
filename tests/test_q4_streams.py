"""Which stream and device torch's own work of a 4-bit cache call goes to (no GPU)."""
import contextlib

import pytest
import torch


@pytest.mark.parametrize("handle,expect", [(0, ("default", 3)), (1, ("default", 3)), (0x7000, ("external", 0x7000, 3)),
                                           (2, ("external", 2, 3))])
def test_stream_handles_are_those_of_the_tensors_device(monkeypatch, handle, expect):
    """A cudaStream_t is taken as a stream of the tensors' device, whatever device is the current one."""
    import decode_attention_append_gb300 as daa
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("default", device))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr, device=None: ("external", ptr, device))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext(s))
    with daa._use_stream(handle, 3) as used:
        assert used == expect
    with daa._use_stream(None, 3) as used:
        assert used is None

    class Stream:  # of another library
        cuda_stream = handle
    with daa._use_stream(Stream(), 3) as used:
        assert used == expect
