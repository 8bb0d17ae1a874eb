"""Which stream a call without one runs on: torch's current one, whatever its private getters say (no GPU: torch's streams
are stood in for)."""

import contextlib

import pytest
import torch

from attention_kv_cache_gb300 import kvsel as K


class Torch:
    """torch's streams: the current one's handle, the public way to it and the private ones."""

    def __init__(self, monkeypatch, device=lambda: 0, raw=None, capturing=False):
        self.now, self.made = 0, 0

        class Stream:
            def __init__(s, handle=None):
                self.made += handle is None
                s.cuda_stream = 1000 + self.made if handle is None else handle

        @contextlib.contextmanager
        def under(stream):
            before, self.now = self.now, stream.cuda_stream
            try:
                yield
            finally:
                self.now = before
        self.under, self.Stream = under, Stream
        monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream(self.now))
        monkeypatch.setattr(torch.cuda, "Stream", Stream)
        monkeypatch.setattr(torch.cuda, "stream", under)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
        monkeypatch.setattr(K, "_current_stream", None)
        for name, f in (("_cuda_getDevice", device), ("_cuda_getCurrentRawStream", raw or (lambda d: self.now))):
            if f == "none":
                monkeypatch.delattr(torch._C, name, raising=False)
            else:
                monkeypatch.setattr(torch._C, name, f, raising=False)


def _follows(t):
    side = t.Stream()
    assert K._stream(None) == t.now == 0
    with t.under(side):
        assert K._stream(None) == side.cuda_stream
    assert K._stream(None) == 0
    assert K._stream(side) == side.cuda_stream and K._stream(7) == 7


def test_torchs_own_getters(monkeypatch):
    _follows(Torch(monkeypatch))


@pytest.mark.parametrize("raw", [lambda d: 0, lambda d: None, lambda d, more: 0, "none"])
def test_getters_that_do_not_follow_the_current_stream(monkeypatch, raw):
    """One that answers 0 looks right on the default stream alone."""
    _follows(Torch(monkeypatch, raw=raw))


def test_no_device_getter(monkeypatch):
    _follows(Torch(monkeypatch, device="none"))


def test_a_first_call_in_a_capture_makes_no_stream(monkeypatch):
    t = Torch(monkeypatch, capturing=True)
    assert K._stream(None) == 0 and t.made == 0 and K._current_stream is None
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    _follows(t)
