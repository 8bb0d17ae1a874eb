"""Attention of a batch whose requests share prefixes: what the single-token call gives, and the fp64 definition.

Tolerances are the single-token call's (its test derives them) with the shared rows' weights over e4m3 pools rounded once to fp16
(2^-11 of each), and one more join of two parts in fp32 (8 u of each, inside its 2 u (n + 64)).
"""

import numpy as np
import pytest
import torch

from oracle import paged_oracle as O
from tests import paged_common as C
from tests.test_gpu_paged_attend import Case as Single

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


class Case(Single):
    """groups: [(shared rows, [own rows of each member])]; the members' tables name the same pages for the shared whole pages."""

    def __init__(self, K, cuda, groups, P=16, order="head", window=0, **kw):
        lens = [s + x for s, own in groups for x in own]
        super().__init__(K, cuda, lens, P=P, order=order, window=window, **kw)
        first, starts = 0, [0]
        for s, own in groups:
            for b in range(first + 1, first + len(own)):
                pages = s // P
                self.tables[b, :pages] = self.tables[first, :pages]
                for rows in self.rows:
                    rows[b][:pages * P] = rows[first][:pages * P]
            # (the members' windows may begin at different shared rows: put what any of them sees)
            for pool, rows in zip(self.pools, self.rows):
                least = min(lens[first:first + len(own)], default=0)
                low = max(0, least - window) if window else 0
                if own:
                    C.put_rows(pool, order, self.tables, P, first, low, rows[first][low:])
            first += len(own)
            starts.append(first)
        self.t = torch.from_numpy(self.tables).to(torch.int32).to(cuda)
        self.indptr = torch.tensor(starts, dtype=torch.int64, device=cuda)
        self.shared = torch.tensor([s for s, _ in groups], dtype=torch.int64, device=cuda)
        self.ws = C.workspace(K, K.kvsel_prefix_attend_workspace_size(self.desc, self.p, len(groups)), cuda)

    def run(self, stream=None):
        self.K.kvsel_prefix_attend(self.desc, self.p, self.q, self.pools[0], self.pools[1], self.t, self.l, self.indptr, self.shared,
                                   self.slopes, self.scales[0], self.scales[1], self.o, self.lse, self.ws, stream=stream)
        return self

    def check(self, error=None):
        torch.cuda.synchronize()
        assert self.K.kvsel_read_device_error(self.ws) == (self.K.OK if error is None else error)
        got, lse, q = C.f64(self.o), C.f64(self.lse), C.f64(self.q)
        eps, w = torch.finfo(C.DT[self.dtype]).eps, 2.0 ** -11 if self.cache == "e4m3" else 2.0 ** -17
        for b, n in enumerate(self.lens):
            for h in range(self.h_kv):
                hs = slice(h * self.G, (h + 1) * self.G)
                k, v = (C.f64(r[b][:n, h]) * (1.0 if s is None else float(s[h])) for r, s in zip(self.rows, self.scales))
                sl = None if self.slopes is None else C.f64(self.slopes)[hs]
                o, ls, mass, zmax = O.paged_attend(q[b, hs], k, v, self.scale, self.softcap, self.window, sl)
                if n == 0:
                    assert (got[b, hs] == 0).all() and np.isneginf(lse[b, hs]).all()
                    continue
                bias = 0.0 if sl is None else float(sl.max()) * min(n, self.window or n)
                dz = 2 * U * ((self.d + 8) * zmax + 4 * self.softcap + 4 * bias)
                if self.cache == "e4m3":
                    dz += U * self.d * self.scale * np.abs(q[b, hs]).max() * np.abs(k).max()
                low = 2 * U * n * np.abs(v).max() if self.cache != "bf16" else 0.0
                tol = eps / 2 * np.abs(o) + (2 * (dz + 2.0 ** -17 + 2 * U * (n + 64)) + w) * mass + low
                bad = ~(np.abs(got[b, hs] - o) <= tol)
                assert not bad.any(), (b, h, bad.sum(), np.argwhere(bad)[0], got[b, hs][bad][0], o[bad][0])
                bad = ~(np.abs(lse[b, hs] - ls) <= dz + 2.0 ** -19 * (1 + np.abs(ls)) + 2 * U * (n + 64))
                assert not bad.any(), (b, h, np.argwhere(bad)[0])
        return self


@pytest.fixture(scope="module")
def K():
    from attention_kv_cache_gb300 import kvsel
    return kvsel


@pytest.mark.parametrize("groups", [
    [(512, [1, 30, 17, 4])], [(16, [1])], [(15, [3, 4])], [(0, [0, 5, 100])], [(4000, [7] * 3)], [(130, [0, 0, 1])],
    [(500, [20, 1]), (0, [9]), (77, []), (1000, [3, 3, 3]), (128, [64])], [(256, [40] * 40)], [(300, [2] * 70)],
    [(100, [1])] * 30, [(0, [0, 0])],
], ids=range(11))
def test_groups(cuda, K, groups):
    """From a group of one to more rows than two tiles, shared lengths that end inside a page, empty groups and requests."""
    Case(K, cuda, groups).run().check()


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("order,P,d", [("head", 16, 128), ("row", 24, 64), ("row", 7, 128), ("head", 5, 64), ("row", 64, 128)])
def test_pools(cuda, K, dtype, cache, order, P, d):
    Case(K, cuda, [(700, [20, 1, 33]), (60, [5] * 40)], dtype=dtype, cache=cache, order=order, P=P, d=d).run().check()


@pytest.mark.parametrize("kw", [
    dict(G=1, h_kv=4), dict(G=5, h_kv=1), dict(G=7, d=64), dict(G=16, h_kv=1), dict(G=8, q_pad=3), dict(softcap=30.0),
    dict(slopes=True), dict(window=1), dict(window=50), dict(window=300, slopes=True), dict(window=600, softcap=10.0, cache="e4m3"),
    dict(window=250, dtype="f16", P=9), dict(scale=0.4, slopes=True, d=64),
], ids=str)
def test_heads_and_masks(cuda, K, kw):
    """Windows that end before, inside and behind the shared rows, at other rows for each member."""
    Case(K, cuda, [(500, [1, 100, 40]), (200, [30, 210])], **kw).run().check()


def test_what_the_single_call_gives(cuda, K):
    """Shared or not, the same attention: within the two calls' tolerances of one another, and equal without shared rows."""
    c = Case(K, cuda, [(800, [3, 60]), (0, [500])]).run()
    torch.cuda.synchronize()
    o, lse = c.o.clone(), c.lse.clone()
    Single.run(c)
    torch.cuda.synchronize()
    assert (lse - c.lse).abs().max() < 1e-5
    assert torch.equal(o[2], c.o[2])
    assert ((o.float() - c.o.float()).abs() <= 2.0 ** -7 * c.o.float().abs() + 1e-5).all()


@pytest.mark.parametrize("what", ["falls", "short", "long", "group"])
def test_bad_groups_are_read_as_unshared(cuda, K, what):
    """Groups that cannot be are reported, and the output is right all the same."""
    c = Case(K, cuda, [(320, [10, 4]), (160, [7, 9])])
    if what == "falls":
        c.indptr[1] = 5
    elif what == "short":
        c.indptr[2] = 3
    elif what == "long":
        c.shared[0] = 325                                         # more than the second member holds
    else:
        c.shared[1] = -1
    c.run().check(error=K.ERR_INVALID_ARG)


def test_rows_that_no_member_sees_may_hold_anything(cuda, K):
    """Infinities and NaN before the shortest member's window, and between the members' windows, stay where they are seen."""
    c = Case(K, cuda, [(400, [1, 200])], window=300, G=4)
    # row 150: seen by the first member (101 .. 401), not by the second (300 .. 600)
    for x, col in ((float("inf"), 3), (float("nan"), 5)):
        v = c.rows[1][0][150:151].clone()
        v[..., col] = x
        C.put_rows(c.pools[1], c.order, c.tables, c.P, 0, 150, v)
        c.run()
        torch.cuda.synchronize()
        seen, unseen = C.f64(c.o)[0][..., col], C.f64(c.o)[1]
        assert (np.isnan(seen) if x != x else seen == x).all() and np.isfinite(unseen).all()


def test_bad_shared_page_is_left_out(cuda, K):
    c = Case(K, cuda, [(160, [5, 6])])
    c.t[0, 3] = c.n_pages + 9
    c.run()
    torch.cuda.synchronize()
    assert K.kvsel_read_device_error(c.ws) == K.ERR_DEVICE
    keep = [t for t in range(166) if not 48 <= t < 64]
    for b, n in enumerate(c.lens):
        mine = [t for t in keep if t < n]
        o = O.paged_attend(C.f64(c.q)[b, :c.G], C.f64(c.rows[0][b][mine, 0]), C.f64(c.rows[1][b][mine, 0]), c.scale)[0]
        assert np.abs(C.f64(c.o)[b, :c.G] - o).max() < 0.02


def test_streams_capture_and_a_shared_workspace(cuda, K):
    """Captured twice over one workspace, with other lengths and groups in a replay."""
    c = Case(K, cuda, [(320, [10, 4]), (160, [7, 9])])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.run(stream=side)
    side.synchronize()
    c.check()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for i, (l, s) in enumerate((([330, 324, 167, 169], [320, 160]), ([321, 320, 160, 165], [160, 0]), ([330, 322, 161, 160], [0, 160]))):
        c.l.copy_(torch.tensor(l))
        c.shared.copy_(torch.tensor(s))
        c.lens = l
        c.o.fill_(7), c.lse.fill_(7)
        graphs[i % 2].replay()
        c.check()
