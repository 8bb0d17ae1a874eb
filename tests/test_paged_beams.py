"""PagedDecoder's beams on the host: what a refused reordering leaves, with the library's calls acted out in place of run (no GPU)."""

import pytest
import torch

from attention_kv_cache_gb300 import kvsel as K
from oracle import paged_oracle as O
from tests.test_paged_decoder import Recorder, Stream, decoder


class Beams(Recorder):
    """kvsel_beam_reorder by its definition: nothing is written where it refuses."""

    def __init__(self, monkeypatch):
        super().__init__(monkeypatch)
        monkeypatch.setattr(K, "kvsel_prefix_attend_workspace_size", lambda cache, desc, groups: 256 * groups)
        monkeypatch.setattr(K, "kvsel_chunk_attend_workspace_size", lambda cache, desc: 256)
        monkeypatch.setattr(K, "kvsel_beam_reorder", self.reorder)
        self.refused = 0

    def reorder(self, cache, desc, parents, lens, tables, queue, head, tables_out, lens_out, head_out, k, v, ws, stream=None):
        self.log.append(("kvsel_beam_reorder", self.now.name, (stream or self.now).name))
        ok = bool(((parents >= 0) & (parents < desc.beams)).all() and (lens >= 0).all())
        out = O.beam_reorder(cache.page_size, parents.tolist(), lens.tolist(), tables.tolist(), queue.tolist(), int(head)) if ok else None
        if out is None:
            self.refused += 1
            return
        for to, x in zip((tables_out, lens_out, queue), out[:3]):
            to.copy_(torch.from_numpy(x))
        head_out.fill_(out[3])


def beams(**kw):
    return decoder(**{**dict(batch=4, beams=2, max_rows=64, n_pages=20), **kw})


def test_offsets_follow_the_lengths(monkeypatch):
    r = Beams(monkeypatch)
    dec = beams()
    dec.lens.copy_(torch.tensor([16, 32, 16, 48]))
    dec.pos_offset.copy_(torch.tensor([1, 2, 3, 4]))
    dec.free_head.fill_(9)
    dec.tables[:, :3] = torch.arange(12, dtype=torch.int32).view(4, 3)
    dec.reorder(torch.tensor([[1, 0], [1, 1]], dtype=torch.int32))
    assert dec.lens.tolist() == [32, 16, 48, 48] and dec.pos_offset.tolist() == [2, 1, 4, 4]
    assert r.refused == 0 and dec.free_head.tolist() == [8]


@pytest.mark.parametrize("what", ["parent", "negative parent", "length", "queue"])
def test_a_refused_reordering_leaves_everything(monkeypatch, what):
    r = Beams(monkeypatch)
    dec = beams()
    dec.lens.copy_(torch.tensor([17, 33, 18, 19]))
    dec.pos_offset.copy_(torch.tensor([1, 2, 3, 4]))
    dec.free_head.fill_(9)
    dec.tables[:, :3] = torch.arange(12, dtype=torch.int32).view(4, 3)
    parents = torch.tensor([[1, 0], [0, 1]], dtype=torch.int32)
    if what == "parent":
        parents[1, 0] = 2
    elif what == "negative parent":
        parents[0, 0] = -1
    elif what == "length":
        dec.lens[3] = -1
    else:
        dec.free_head.fill_(21)
    names = ("lens", "pos_offset", "free_head", "tables", "free_pages")
    before = {x: getattr(dec, x).clone() for x in names}
    dec.reorder(parents)
    assert r.refused == 1
    for x in names:
        assert torch.equal(getattr(dec, x), before[x]), x


def test_a_refused_fork_shares_what_was_shared(monkeypatch):
    r = Beams(monkeypatch)
    dec = beams()
    dec.lens.copy_(torch.tensor([40, 0, 17, 0]))
    dec.free_head.fill_(9)
    dec.tables[:, :3] = torch.arange(12, dtype=torch.int32).view(4, 3)
    dec.fork()
    assert r.refused == 0 and dec.fork_rows.tolist() == [32, 16] and dec.lens.tolist() == [40, 40, 17, 17]
    dec.lens += 30
    dec.free_head.fill_(21)
    dec.fork()
    assert r.refused == 1 and dec.fork_rows.tolist() == [32, 16]
    fresh = beams()
    fresh.lens.copy_(torch.tensor([40, 40, 40, 40]))
    fresh.free_head.fill_(21)
    fresh.fork()
    assert r.refused == 2 and fresh.fork_rows.tolist() == [0, 0]


def test_a_reordering_is_one_streams_work(monkeypatch):
    r = Beams(monkeypatch)
    dec = beams()
    side = Stream("side", r.log)
    r.log.clear()
    dec.reorder(torch.zeros(2, 2, dtype=torch.int32), stream=side)
    dec.fork(stream=side)
    assert r.log[0] == ("wait", "side", "main") and all(e[1] == "side" for e in r.log), r.log


def test_errors_of_outgrown_workspaces_are_found(monkeypatch):
    """A captured step goes on writing its errors where it did."""
    Beams(monkeypatch)
    errors = {}
    monkeypatch.setattr(K, "kvsel_read_device_error", lambda ws, stream=None: errors.pop(ws.data_ptr(), K.OK))
    dec = decoder(batch=4)
    small = dec.ws
    long = lambda *x: torch.tensor(x)              # noqa: E731
    dec.share(long(0, 2, 3, 4), long(16, 0, 0))
    if dec.ws is small:                            # (the workspace is larger than this one's need)
        monkeypatch.setattr(K, "kvsel_prefix_attend_workspace_size", lambda cache, desc, groups: small.numel() + 256)
        dec.share(long(0, 2, 4), long(16, 0))
    assert dec.ws is not small and dec.device_error() == K.OK
    errors[small.data_ptr()] = K.ERR_DEVICE
    assert dec.device_error() == K.ERR_DEVICE and dec.device_error() == K.OK
    errors.update({small.data_ptr(): K.ERR_INVALID_ARG, dec.ws.data_ptr(): K.ERR_DEVICE})
    assert dec.device_error() == K.ERR_INVALID_ARG and dec.device_error() == K.OK


def test_a_larger_workspace_begins_on_the_stream(monkeypatch):
    r = Beams(monkeypatch)
    monkeypatch.setattr(torch, "zeros", r.made("zeros", torch.zeros))
    dec = decoder(batch=4)
    monkeypatch.setattr(K, "kvsel_prefix_attend_workspace_size", lambda cache, desc, groups: dec.ws.numel() + 256)
    side = Stream("side", r.log)
    r.log.clear()
    dec.share(torch.tensor([0, 4]), torch.tensor([16]), stream=side)
    assert r.log == [("zeros", "side")]


@pytest.mark.parametrize("way", ["chunk", "admit"])
def test_replaced_prompts_share_no_rows(monkeypatch, way):
    """Rows that a set's beams hold no more are not shared when new ones come in; what other sets share stays."""
    r = Beams(monkeypatch)
    dec = beams(max_tokens=100)
    dec.lens.copy_(torch.tensor([40, 0, 33, 0]))
    dec.free_head.fill_(9)
    dec.tables[:, :3] = torch.arange(12, dtype=torch.int32).view(4, 3)
    dec.fork()
    assert dec.fork_rows.tolist() == [32, 32]
    side = Stream("side", r.log)

    def come():
        r.log.clear()
        if way == "chunk":
            dec.begin_chunk(torch.tensor([5, 6, 7, 8]), stream=side)
        else:
            dec.admit(*(torch.zeros(4, 2, 2, 3, 64, dtype=torch.bfloat16) for _ in range(2)), [50, 50, 50, 50], stream=side)
        assert [e[2] for e in r.log if e[0] == "kvsel_page_assign"] == ["side"]

    come()
    assert dec.fork_rows.tolist() == [32, 32]
    dec.lens[:2] = torch.tensor([50, 0])                       # one of the set's beams begins anew
    come()
    assert dec.fork_rows.tolist() == [0, 32]
