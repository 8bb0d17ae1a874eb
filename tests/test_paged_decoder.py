"""PagedDecoder on the host: the order of its work between streams and its checks, with the library's calls recorded in
place of run (no GPU)."""

import contextlib

import pytest
import torch

from attention_kv_cache_gb300 import kvsel as K
from attention_kv_cache_gb300 import pipeline


class Stream:
    def __init__(self, name, log):
        self.name, self.log, self.cuda_stream = name, log, id(self)

    def wait_stream(self, other):
        self.log.append(("wait", self.name, other.name))


class Recorder:
    """Streams and the library's calls; `at` notes what is done under which current stream."""

    def __init__(self, monkeypatch):
        self.log = []
        self.main = Stream("main", self.log)
        self.now = self.main
        cuda = torch.cuda
        monkeypatch.setattr(cuda, "current_stream", lambda device=None: self.now)
        monkeypatch.setattr(cuda, "stream", self.under)
        monkeypatch.setattr(K, "kvsel_paged_attend_workspace_size", lambda cache, desc: 256)
        for name in ("kvsel_page_assign", "kvsel_rope_append", "kvsel_paged_attend"):
            monkeypatch.setattr(K, name, self.call(name))
        for name in ("empty", "full_like"):
            monkeypatch.setattr(torch, name, self.made(name, getattr(torch, name)))

    @contextlib.contextmanager
    def under(self, stream):
        before, self.now = self.now, stream
        try:
            yield
        finally:
            self.now = before

    def call(self, name):
        return lambda *a, stream=None, **kw: self.log.append((name, self.now.name, (stream or self.now).name, a))

    def made(self, name, f):
        def wrapped(*a, **kw):
            self.log.append((name, self.now.name))
            return f(*a, **kw)
        return wrapped


def decoder(**kw):
    base = dict(n_layers=2, h_q=8, h_kv=2, head_dim=64, batch=3, max_rows=48, n_pages=12, page_size=16, device="cpu")
    return pipeline.PagedDecoder(**{**base, **kw})


def caches(rows=20, batch=3, n_layers=2, h_kv=2, d=64, dtype=torch.bfloat16):
    return tuple(torch.zeros(batch, n_layers, h_kv, rows, d, dtype=dtype) for _ in range(2))


def test_admission_is_one_streams_work(monkeypatch):
    """Counts, offsets, slots and kernels all on the stream that is given, behind the current one."""
    r = Recorder(monkeypatch)
    dec = decoder()
    side = Stream("side", r.log)
    r.log.clear()
    dec.admit(*caches(), [30, 31, 32], stream=side)
    assert r.log[0] == ("wait", "side", "main")
    assert all(e[1] == "side" for e in r.log), r.log
    calls = [e for e in r.log if e[0].startswith("kvsel")]
    assert [e[0] for e in calls] == ["kvsel_page_assign"] + 6 * ["kvsel_rope_append"]
    assert all(e[2] == "side" for e in calls)
    assert {e[0] for e in r.log} >= {"empty", "full_like"}
    r.log.clear()
    dec = decoder()
    r.log.clear()
    dec.admit(*caches(), [30, 31, 32])
    assert all(e[1] == "main" for e in r.log)
