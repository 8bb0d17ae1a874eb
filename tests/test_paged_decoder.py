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


def step_rows(n=3, h_q=8, h_kv=2, d=64, dtype=torch.bfloat16):
    return [torch.zeros(n, h, d, dtype=dtype) for h in (h_q, h_kv, h_kv)]


@pytest.mark.parametrize("at,shape,dtype", [
    (0, (4, 8, 64), torch.bfloat16), (0, (2, 8, 64), torch.bfloat16), (0, (3, 9, 64), torch.bfloat16),
    (0, (3, 8, 128), torch.bfloat16), (0, (3, 8, 64), torch.float16), (0, (3, 8 * 64), torch.bfloat16),
    (1, (4, 2, 64), torch.bfloat16), (1, (3, 1, 64), torch.bfloat16), (1, (3, 2, 32), torch.bfloat16),
    (1, (3, 2, 64), torch.float32), (2, (4, 2, 64), torch.bfloat16), (2, (3, 1, 64), torch.bfloat16)])
def test_rows_of_another_batch_are_refused(monkeypatch, at, shape, dtype):
    """More rows than the batch has would be read past its slots and written past its queries."""
    r = Recorder(monkeypatch)
    dec = decoder()
    x = step_rows()
    r.log.clear()
    dec.layer(0, *x)
    assert [e[0] for e in r.log] == ["kvsel_rope_append", "kvsel_paged_attend"]
    r.log.clear()
    x[at] = torch.zeros(shape, dtype=dtype)
    with pytest.raises(ValueError):
        dec.layer(0, *x)
    x[at] = torch.zeros(step_rows()[at].shape, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError):
        dec.layer(0, *x)
    assert not any(e[0].startswith("kvsel") for e in r.log)


@pytest.mark.parametrize("kw", [dict(batch=4), dict(batch=2), dict(n_layers=1), dict(h_kv=1), dict(d=32),
                                dict(dtype=torch.float16)])
def test_caches_of_another_shape_are_refused(monkeypatch, kw):
    r = Recorder(monkeypatch)
    dec = decoder()
    good, bad = caches(), caches(**kw)
    r.log.clear()
    for pair in (bad, (good[0], bad[1]), (bad[0], good[1])):
        with pytest.raises(ValueError):
            dec.admit(*pair, [30, 31, 32])
    assert not any(e[0].startswith("kvsel") for e in r.log)


def test_admission_checks_rows_and_texts(monkeypatch):
    r = Recorder(monkeypatch)
    dec = decoder()
    r.log.clear()
    for rows in (-1, 21):
        with pytest.raises(ValueError):
            dec.admit(*caches(), [30, 31, 32], rows=rows)
    for text in ([30, 31], [30, 31, 32, 33], [[30, 31, 32]], 30):
        with pytest.raises(ValueError):
            dec.admit(*caches(), text)
    with pytest.raises(ValueError):
        dec.admit(caches(rows=20)[0], caches(rows=19)[1], [30, 31, 32])
    assert not any(e[0].startswith("kvsel") for e in r.log)
    dec.admit(*caches(), [30, 31, 32], rows=7)
    assert sum(e[0] == "kvsel_rope_append" for e in r.log) == 6


@pytest.mark.parametrize("kw", [dict(window=16), dict(slopes=torch.ones(8)), dict(window=16, slopes=torch.ones(8))])
def test_a_window_over_a_compacted_cache_is_refused(monkeypatch, kw):
    """It would count kept rows, not the positions of the text they were kept from."""
    r = Recorder(monkeypatch)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    dec = decoder(**kw)
    for text in ([30, 31, 32], [20, 20, 21], torch.tensor([20, 19, 20])):
        r.log.clear()
        with pytest.raises(ValueError):
            dec.admit(*caches(), text)
        assert not any(e[0].startswith("kvsel") for e in r.log)
    dec.admit(*caches(), [20, 20, 20])                       # whole texts
    assert sum(e[0] == "kvsel_rope_append" for e in r.log) == 6
    dec.lens += 25                                           # (20 rows, and 5 steps since)
    dec.admit(*caches(), [45, 45, 45])
    with pytest.raises(ValueError):
        dec.admit(*caches(), [46, 45, 45])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(ValueError):
        dec.admit(*caches(), [45, 45, 45])
    plain = decoder()
    plain.admit(*caches(), [30, 31, 32])                     # and neither: any text, in a capture too
