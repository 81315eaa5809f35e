"""How the tensor helpers call the library, on the CPU: the library's part is
replaced, what is looked at is the Python around it."""
import contextlib

import pytest

torch = pytest.importorskip("torch")
from monarch_block_diagonal_amd import torch_api as T  # noqa: E402


class Streams:
    """Stands in for torch.cuda's streams: a handle that is 0 makes a new stream of a raw one, as in torch."""

    def __init__(self, monkeypatch):
        self.current = [0]
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle if handle else 0xbad)
        monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: 0)
        monkeypatch.setattr(torch.cuda, "stream", self.enter)

    @contextlib.contextmanager
    def enter(self, stream):
        self.current.append(stream)
        yield
        self.current.pop()


@pytest.mark.parametrize("handle", [0, 0x7f0040])
def test_a_raw_stream_is_the_one_named(monkeypatch, handle):
    streams = Streams(monkeypatch)
    streams.current = [0x1234]   # the caller's current stream is another one
    assert T._on_stream(handle, lambda: streams.current[-1]) == handle
