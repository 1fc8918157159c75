"""Streams in the Python binding, without a GPU: torch's stream functions are replaced by
ones that only note which stream is current when memory is made."""
import contextlib

import pytest
import torch

import w4a16_dequant_gemm_amd as w4

CURRENT = 0x10


class Streams:
    """Stands in for torch's current stream: a stack of handles."""

    def __init__(self, monkeypatch):
        self.stack, self.made = [CURRENT], []
        monkeypatch.setattr(torch.cuda, "ExternalStream",
                            lambda handle, device=None: ("external", handle, device))
        monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("default", 0, device))
        monkeypatch.setattr(torch.cuda, "stream", self.use)
        zeros = torch.zeros

        def noted(*shape, dtype=None, device=None):
            self.made.append(("zeros", self.stack[-1]))
            return zeros(*shape, dtype=dtype)
        monkeypatch.setattr(torch, "zeros", noted)
        monkeypatch.setattr(w4, "_workspaces", {})
        monkeypatch.setattr(w4, "_retired_workspaces", [])

    @contextlib.contextmanager
    def use(self, stream):
        self.stack.append(stream[1])
        yield
        self.stack.pop()


@pytest.fixture
def streams(monkeypatch):
    return Streams(monkeypatch)


@pytest.mark.parametrize("handle", [CURRENT, 0x20, 0])
def test_workspace_is_filled_on_the_stream_that_uses_it(streams, handle):
    ws = w4._workspace_at(1 << 20, 0, handle)
    assert streams.made == [("zeros", handle)]
    assert w4._workspace_at(1 << 20, 0, handle) is ws
    w4._workspace_at((1 << 20) + 1, 0, handle)        # grows
    assert streams.made == [("zeros", handle)] * 2
