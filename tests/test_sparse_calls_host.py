"""Host-side checks of how the sparse-attention and gradient calls reach the
device (no GPU needed): the stream they launch on, what they refuse, and what
their kernels may not do."""
import contextlib

import pytest
import torch

from tests.test_abi_host import L  # noqa: F401  (fixture)
from tests.test_sparse_host import _Pretend


@pytest.mark.parametrize("handle,want", [(0, 0), (1, 1), (0x7f00, 0x7f00)])
def test_a_stream_handle_launches_on_that_stream(monkeypatch, handle, want):
    """Handle 0 is the default stream.  torch takes an ExternalStream of 0 for one
    without a handle and makes a stream of its own, on which the kernels would run
    beside the work that produces their inputs."""
    import spacetime_attention_vdit_b200 as vd

    class Stream:
        def __init__(self, cuda_stream):
            self.cuda_stream = cuda_stream

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h: Stream(h if h else 0xbad))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "stream", contextlib.nullcontext)
    context, got = vd._launch_stream(_Pretend(1, 200, 2, 32), "q", handle)
    assert got == want
    with context as st:
        assert st.cuda_stream == want            # what the call allocates belongs to the same stream
