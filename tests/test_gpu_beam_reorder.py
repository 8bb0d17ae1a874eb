"""The beams' pages after a selection, against the definition with lists: tables, lengths, queue, and every byte of the pools."""

import numpy as np
import pytest
import torch

from oracle import paged_oracle as O
from tests import paged_common as C

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


class Case:
    """sets of beams whose tables share pages as a search leaves them; lens[s] rows of every beam of set s."""

    def __init__(self, K, cuda, lens, beams, P=16, h_kv=2, d=64, layers=2, cache="bf16", order="head", seed=0, spare=None, extra=2,
                 in_place=True, ragged=False):
        rng = np.random.default_rng(seed)
        self.K, self.P, self.beams, self.order, self.cuda, self.in_place = K, P, beams, order, cuda, in_place
        sets = len(lens)
        self.lens = np.array([n if not ragged else int(rng.integers(0, n + 1)) for n in lens for _ in range(beams)])
        self.max_blocks = max(1, max(-(-n // P) for n in lens) + extra)
        rows, used = [], 0
        for s in range(sets):
            share = [rng.integers(0, i + 1, beams).tolist() for i in range(3)]
            pages = {}
            for k in range(beams):
                n = -(-int(self.lens[s * beams + k]) // P)
                r = []
                for c in range(self.max_blocks):
                    if c >= n:
                        r.append(-9)
                        continue
                    # old columns are the set's, the next ones shared by some, the last a beam's own
                    owner = 0 if c < n - 3 else k if c == n - 1 or ragged else share[min(2, n - 1 - c)][k]
                    key = (c, owner) if not ragged or c < 1 else (c, k, "own")
                    if key not in pages:
                        pages[key] = used
                        used += 1
                    r.append(pages[key])
                rows.append(r)
        spare = sets * beams + 3 if spare is None else spare
        self.n_pages = used + spare
        ids = rng.permutation(self.n_pages)
        self.tables = np.array([[ids[x] if x >= 0 else x for x in r] for r in rows])
        self.queue, self.head = np.concatenate([np.full(used, -1), ids[used:]]), used
        dt = DT[cache]
        shape = (layers, self.n_pages, h_kv, P, d) if order == "head" else (layers, self.n_pages, P, h_kv, d)
        self.pools = [torch.randint(0, 255, shape + (dt.itemsize,), generator=torch.Generator().manual_seed(seed), dtype=torch.uint8)
                      .to(cuda).view(dt)[..., 0] if dt.itemsize == 1 else
                      torch.randint(0, 30000, shape, generator=torch.Generator().manual_seed(seed + i), dtype=torch.int16).to(cuda).view(dt)
                      for i in range(2)]
        kinds = C.kinds(K)
        self.desc = K.make_cache_desc(h_q=h_kv, h_kv=h_kv, head_dim=d, page_size=P, n_pages=self.n_pages,
                                      dtype=kinds["bf16" if cache == "e4m3" else cache], cache_dtype=kinds[cache],
                                      order=K.ORDER_HEAD if order == "head" else K.ORDER_ROW)
        self.p = K.make_beam_reorder_desc(batch=sets, beams=beams, max_blocks=self.max_blocks, n_layers=layers,
                                          layer_stride=self.pools[0].stride(0))
        self.ws = C.workspace(K, K.kvsel_beam_reorder_workspace_size(self.p), cuda)
        i64, i32 = dict(dtype=torch.int64, device=cuda), dict(dtype=torch.int32, device=cuda)
        self.t, self.f = torch.tensor(self.tables, **i32), torch.tensor(self.queue, **i32)
        self.l, self.h = torch.tensor(self.lens, **i64), torch.tensor([self.head], **i64)
        if in_place:
            self.to, self.lo, self.ho = self.t, self.l, self.h
        else:
            self.to, self.lo, self.ho = torch.full_like(self.t, -9), torch.full_like(self.l, -5), torch.full_like(self.h, -5)

    def run(self, parents, stream=None):
        self.parents = torch.tensor(parents, dtype=torch.int32, device=self.cuda) if not torch.is_tensor(parents) else parents
        self.before = [x.view(torch.uint8).clone() if x.element_size() == 1 else x.clone() for x in self.pools]
        self.K.kvsel_beam_reorder(self.desc, self.p, self.parents, self.l, self.t, self.f, self.h, self.to, self.lo, self.ho,
                                  self.pools[0], self.pools[1], self.ws, stream=stream)
        return self

    def check(self, error=None):
        torch.cuda.synchronize()
        assert self.K.kvsel_read_device_error(self.ws) == (self.K.OK if error is None else error)
        held = [x.view(torch.uint8) if x.element_size() == 1 else x for x in self.pools]
        ref = None if error else O.beam_reorder(self.P, self.parents.tolist(), self.lens, self.tables, self.queue, self.head)
        if ref is None:
            assert all(torch.equal(a, b) for a, b in zip(held, self.before))
            if not self.in_place:
                assert (self.lo == -5).all() and (self.ho == -5).all() and (self.to == -9).all()
            else:
                assert np.array_equal(self.t.cpu().numpy(), self.tables) and np.array_equal(self.l.cpu().numpy(), self.lens)
            assert np.array_equal(self.f.cpu().numpy(), self.queue)
            return self
        tables, lens, queue, head, copies = ref
        assert np.array_equal(self.lo.cpu().numpy(), lens) and int(self.ho) == head
        assert np.array_equal(self.f.cpu().numpy(), queue)
        held_cols = np.arange(self.max_blocks) < -(-lens // self.P)[:, None]
        got = self.to.cpu().numpy()
        assert np.array_equal(got[held_cols], tables[held_cols])
        if self.in_place:
            assert np.array_equal(got[~held_cols], self.tables[~held_cols])
        else:
            assert (got[~held_cols] == -9).all()
        for pool, old in zip(held, self.before):
            want = old.clone()
            view, source = (x if self.order == "row" else x.transpose(2, 3) for x in (want, old))      # [layer, page, row, ...]
            for _, _, a, b, n in copies:
                view[:, b, :n] = source[:, a, :n]
            assert torch.equal(pool, want)
        self.tables, self.lens, self.queue, self.head = tables, lens, queue, head
        if self.in_place:
            assert np.array_equal(got[held_cols], tables[held_cols])
            self.tables = got
        # a page is named or in the queue, never both, and never in two places of the queue
        free = queue[head:]
        named = set(got[held_cols].tolist())
        assert len(set(free.tolist())) == len(free) and not named & set(free.tolist())
        return self


@pytest.fixture(scope="module")
def K():
    from attention_kv_cache_gb300 import kvsel
    return kvsel


def _parents(rng, sets, beams, kept):
    out = []
    for _ in range(sets):
        chosen = rng.permutation(beams)[:max(1, kept)]
        out.append(rng.permutation(np.concatenate([chosen, rng.choice(chosen, beams - len(chosen))])).tolist())
    return out


@pytest.mark.parametrize("beams,lens", [(1, [40]), (2, [1]), (2, [16, 17]), (4, [100]), (4, [0, 33, 5000]), (8, [77] * 20),
                                        (64, [50, 200]), (5, [2049, 128, 127])])
@pytest.mark.parametrize("in_place", [True, False])
def test_steps_on_from_one_another(cuda, K, beams, lens, in_place):
    rng = np.random.default_rng(beams)
    for kept in {1, max(1, beams // 2), beams}:
        c = Case(K, cuda, lens, beams, seed=kept, in_place=in_place)
        for step in range(3 if in_place else 1):
            c.run(_parents(rng, len(lens), beams, kept)).check()


@pytest.mark.parametrize("cache,order,P,h_kv,d", [("bf16", "head", 16, 2, 128), ("f16", "row", 24, 3, 64), ("e4m3", "head", 7, 2, 128),
                                                  ("e4m3", "row", 33, 4, 16), ("bf16", "row", 1, 1, 256), ("f16", "head", 256, 1, 48)])
def test_pools(cuda, K, cache, order, P, h_kv, d):
    rng = np.random.default_rng(3)
    c = Case(K, cuda, [5 * P + P // 2, 3 * P + 1], 4, P=P, h_kv=h_kv, d=d, cache=cache, order=order, layers=3)
    for _ in range(2):
        c.run(_parents(rng, 2, 4, 2)).check()


def test_beams_of_different_lengths(cuda, K):
    rng = np.random.default_rng(4)
    for seed in range(4):
        c = Case(K, cuda, [100, 300], 6, seed=seed, ragged=True, in_place=False)
        c.run(_parents(rng, 2, 6, 3)).check()


def test_fork_of_a_prompt(cuda, K):
    """All parents 0, the other beams empty: whole pages are shared, the part-full one copied from the queue."""
    for n in (0, 16, 37):
        c = Case(K, cuda, [n], 4)
        c.lens[1:] = 0
        c.l[1:] = 0
        owned = set(c.tables[0][:-(-n // 16)].tolist())
        free = [p for p in range(c.n_pages) if p not in owned]
        c.queue, c.head = np.array([-1] * len(owned) + free), len(owned)
        c.f = torch.tensor(c.queue, dtype=torch.int32, device=cuda)
        c.h.fill_(c.head)
        c.run([[0, 0, 0, 0]]).check()


@pytest.mark.parametrize("what", ["parent", "negative parent", "length", "page", "queue", "head", "queue page"])
@pytest.mark.parametrize("in_place", [True, False])
def test_what_cannot_be_carried_out_changes_nothing(cuda, K, what, in_place):
    c = Case(K, cuda, [40, 50], 3, spare=0 if what == "queue" else None, in_place=in_place)
    parents, error = [[0, 0, 1], [2, 1, 0]], K.ERR_INVALID_ARG
    if what == "parent":
        parents[1][2] = 3
    elif what == "negative parent":
        parents[0][0] = -1
    elif what == "length":
        c.l[4] = c.max_blocks * c.P + 1
        c.lens[4] = c.max_blocks * c.P + 1
    elif what == "page":
        c.t[5, 1] = c.n_pages
        c.tables[5, 1] = c.n_pages
        error = K.ERR_DEVICE
    elif what == "queue":
        # twins and nothing freed: beams that hold nothing themselves
        c.lens[1:3] = 0
        c.l[1:3] = 0
        parents = [[0, 0, 0], [0, 1, 2]]
    elif what == "head":
        c.h.fill_(len(c.queue) + 1)
        c.head = len(c.queue) + 1
    else:
        c.lens[1:3] = 0
        c.l[1:3] = 0
        parents, error = [[0, 0, 0], [0, 1, 2]], K.ERR_DEVICE
        c.f[c.head] = -3
        c.queue[c.head] = -3
    c.run(parents).check(error=error)


def test_streams_and_capture(cuda, K):
    rng = np.random.default_rng(6)
    c = Case(K, cuda, [130, 44], 4)
    side = torch.cuda.Stream()
    parents = torch.tensor(_parents(rng, 2, 4, 2), dtype=torch.int32, device=cuda)
    torch.cuda.synchronize()
    c.run(parents, stream=side)
    side.synchronize()
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.K.kvsel_beam_reorder(c.desc, c.p, parents, c.l, c.t, c.f, c.h, c.to, c.lo, c.ho, c.pools[0], c.pools[1], c.ws)
    for kept in (1, 3, 2):
        parents.copy_(torch.tensor(_parents(rng, 2, 4, kept)))
        c.before = [x.clone() for x in c.pools]
        g.replay()
        c.check()
