"""Pages, slots, positions and block tables built on the GPU, against the request-by-request definition (exact)."""

import numpy as np
import pytest
import torch

from oracle import paged_oracle as O
from tests import paged_common as C

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, K, cuda, lens, new, P=16, pad=0, seed=0, head=2, spare=4, offsets=False, max_blocks=None):
        self.K, self.cuda, self.P = K, cuda, P
        rng = np.random.default_rng(seed)
        self.lens, self.new = [int(x) for x in lens], [int(x) for x in new]
        batch = len(lens)
        held = sum(-(-n // P) for n in lens)
        need = sum(-(-(n + m) // P) for n, m in zip(lens, new)) - held
        self.n_pages = held + need + head + spare
        self.max_blocks = max_blocks or max(1, max(-(-(n + m) // P) for n, m in zip(lens, new)) + 1)
        ids = rng.permutation(self.n_pages)
        self.tables = np.full((batch, self.max_blocks), -3, np.int64)
        at = 0
        for b, n in enumerate(lens):
            m = -(-n // P)
            self.tables[b, :m] = ids[at:at + m]
            at += m
        self.free, self.head = ids[at:], head
        self.max_tokens = sum(new) + pad
        self.offsets = rng.integers(0, 10 ** 9, batch) if offsets else None
        i64 = dict(dtype=torch.int64, device=cuda)
        self.d = {"lens": torch.tensor(self.lens, **i64), "new": torch.tensor(self.new, **i64),
                  "free": torch.from_numpy(self.free).to(torch.int32).to(cuda), "head": torch.tensor([head], **i64),
                  "tables": torch.from_numpy(self.tables).to(torch.int32).to(cuda),
                  "lens_out": torch.full((batch,), -9, **i64), "head_out": torch.full((1,), -9, **i64),
                  "indptr": torch.full((batch + 1,), -9, **i64), "slots": torch.full((self.max_tokens,), -9, **i64),
                  "pos": torch.full((self.max_tokens,), -9, **i64),
                  "ids": torch.full((self.max_tokens,), -9, dtype=torch.int32, device=cuda),
                  "off": None if self.offsets is None else torch.from_numpy(self.offsets).to(cuda)}
        self.ws = C.workspace(K, K.kvsel_page_assign_workspace_size(batch), cuda)

    def run(self, in_place=False, stream=None):
        d = self.d
        if in_place:
            d["lens_out"], d["head_out"] = d["lens"], d["head"]
        self.K.kvsel_page_assign(self.P, self.n_pages, d["lens"], d["new"], d["free"], d["head"], d["tables"],
                                 d["lens_out"], d["head_out"], d["indptr"], d["slots"], d["pos"], d["ids"], self.ws,
                                 pos_offset=d["off"], stream=stream)
        return self

    def want(self):
        return O.page_assign(self.P, self.lens, self.new, self.free, self.head, self.tables, self.max_tokens, self.offsets)

    def check(self, error=None):
        torch.cuda.synchronize()
        assert self.K.kvsel_read_device_error(self.ws) == (self.K.OK if error is None else error)
        w, d = self.want(), self.d
        if w is None:
            assert error == self.K.ERR_INVALID_ARG
            w = {"slots": np.full(self.max_tokens, -1), "positions": np.zeros(self.max_tokens),
                 "seq_ids": np.full(self.max_tokens, -1), "lens": np.array(self.lens), "head": self.head,
                 "indptr": np.zeros(len(self.lens) + 1), "tables": self.tables}
        for name, key in (("slots", "slots"), ("positions", "pos"), ("seq_ids", "ids"), ("lens", "lens_out"),
                          ("indptr", "indptr"), ("tables", "tables")):
            if d[key] is not None:
                np.testing.assert_array_equal(d[key].cpu().numpy(), w[name], err_msg=name)
        assert int(d["head_out"]) == w["head"]


SHAPES = [
    dict(lens=[0], new=[1]), dict(lens=[0], new=[0]), dict(lens=[15], new=[1]), dict(lens=[16], new=[1], pad=5),
    dict(lens=[0, 16, 17, 31], new=[1, 1, 0, 40], pad=3, offsets=True), dict(lens=[5, 6, 7], new=[0, 0, 0], pad=9),
    dict(lens=[0] * 7, new=[3] * 7, P=1), dict(lens=[255, 256, 257], new=[1, 1, 600], P=256),
    dict(lens=[100, 0, 3], new=[0, 5000, 0], pad=1), dict(lens=[0, 0, 0, 50], new=[0, 0, 4097, 0]),
    dict(lens=[7, 9], new=[20000, 30001], P=7, pad=777),
    dict(lens=range(0, 4096), new=[1] * 4096, P=16, pad=100), dict(lens=range(0, 4096), new=[0, 1] * 2048, P=3),
    dict(lens=range(3, 1000), new=list(range(997)), P=32, pad=13, offsets=True),
    dict(lens=[1, 0] * 129, new=[0, 1] * 129, P=16),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kw", SHAPES, ids=range(len(SHAPES)))
def test_steps(cuda, kw, in_place):
    from attention_kv_cache_gb300 import kvsel as K
    Case(K, cuda, **kw).run(in_place).check()


def test_nullable_outputs_and_exact_queue(cuda):
    from attention_kv_cache_gb300 import kvsel as K
    for new in ([50, 1], [5000, 1]):
        c = Case(K, cuda, [3, 4], new, spare=0)          # the queue's last page is taken
        c.d["pos"] = c.d["ids"] = None
        c.run().check()
    c = Case(K, cuda, [3, 4], [0, 0])                     # no token at all
    c.run().check()


@pytest.mark.parametrize("big", [1, 5000])
@pytest.mark.parametrize("fault", ["queue", "tokens", "negative length", "negative count", "long", "huge", "head", "head past"])
def test_a_step_that_cannot_be_carried_out_assigns_nothing(cuda, fault, big):
    from attention_kv_cache_gb300 import kvsel as K
    c = Case(K, cuda, [30, 40, 50], [big, 2, 3], spare=0)
    if fault == "queue":
        c.free = c.free[:-1]
        c.d["free"] = c.d["free"][:-1].clone()
    elif fault == "tokens":
        c.max_tokens -= 1
        for k in ("slots", "pos", "ids"):
            c.d[k] = c.d[k][:-1].clone()
    else:
        key, at, value = {"negative length": ("lens", 1, -1), "negative count": ("new", 2, -1),
                          "long": ("new", 1, c.max_blocks * c.P), "huge": ("lens", 0, 2 ** 62),
                          "head": ("head", 0, -1), "head past": ("head", 0, len(c.free) + 1)}[fault]
        c.d[key][at] = value
        if key == "head":
            c.head = value
        else:
            getattr(c, key)[at] = value
    c.run().check(error=K.ERR_INVALID_ARG)
    c.run(in_place=True).check(error=K.ERR_INVALID_ARG)


@pytest.mark.parametrize("big", [20, 5000])
def test_page_ids_outside_the_pool_get_no_slot(cuda, big):
    from attention_kv_cache_gb300 import kvsel as K
    for bad in (-1, None, 2 ** 31 - 1):
        c = Case(K, cuda, [30, 40], [big, 2])
        value = c.n_pages if bad is None else bad
        c.d["free"][c.head] = value                       # request 0's first new page
        c.d["tables"][1, 2] = value                       # request 1's last page, partly filled
        c.free = c.free.copy()
        c.free[c.head] = value
        c.tables[1, 2] = value
        w = c.want()
        c.run()
        torch.cuda.synchronize()
        assert K.kvsel_read_device_error(c.ws) == K.ERR_DEVICE
        lost = np.zeros(c.max_tokens, bool)
        lost[2:18] = True                                 # rows 32 .. 47 of request 0
        lost[big:big + 2] = True                          # rows 40, 41 of request 1
        np.testing.assert_array_equal(c.d["slots"].cpu().numpy(), np.where(lost, -1, w["slots"]))
        np.testing.assert_array_equal(c.d["tables"].cpu().numpy(), w["tables"])


@pytest.mark.parametrize("big", [1, 4500])
def test_captured_steps_go_on_from_one_another(cuda, big):
    """Replays of one captured in-place step: every one takes the next pages of the queue."""
    from attention_kv_cache_gb300 import kvsel as K
    c = Case(K, cuda, [0, 15, 31, 500], [big, 1, 1, 1], spare=40 + 4 * big // 16, pad=2, max_blocks=1200)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(in_place=True)
    for _ in range(4):
        w = c.want()
        g.replay()
        c.check()
        c.lens, c.head, c.tables = [int(x) for x in w["lens"]], w["head"], w["tables"]


def test_another_stream(cuda):
    from attention_kv_cache_gb300 import kvsel as K
    s = torch.cuda.Stream()
    cases = [Case(K, cuda, [9] * 50, [n] * 50, seed=n) for n in (1, 200)]
    torch.cuda.synchronize()
    for c in cases:
        c.run(stream=s)
    for c in cases:
        c.check()
