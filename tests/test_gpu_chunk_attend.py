"""Attention of many new tokens per request over a paged pool against the fp64 definition.

Rows that no token of a request sees are NaN in the pool (behind its last, before every window, spare pages), and entries of its table
behind its last page are outside the pool.

Tolerances: those of the single-token call (its test derives dz, the error of a score, from u = 2^-24) but for the weights,
each rounded once to the products' type: by at most half a step, w = 2^-8 of it over bf16 and 2^-11 over fp16 products (e4m3 pools
too), with 2^-20 for the exponent taken 13 orders from its own.  The sums are of unrounded weights.  So
    |o - ref| <= eps/2 |ref| + (2 (dz + 2^-20 + 2 u (n + 64)) + w) mass (+ 2 u n max|v|: fp16 weights below its normal range),
    |lse - ref| <= dz + 2^-19 (1 + |ref|) + 2 u (n + 64).
"""

import numpy as np
import pytest
import torch

from oracle import paged_oracle as O
from tests import paged_common as C

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


class Case:
    """Inputs of one call: held[b] rows before the step and new[b] tokens of each request, `pad` tokens behind them."""

    def __init__(self, K, cuda, held, new, h_kv=2, G=4, d=128, P=16, dtype="bf16", cache=None, order="head", softcap=0.0, window=0,
                 slopes=False, scale=0.0, seed=0, spare=3, pad=3, q_pad=0, strides=None, fill=-7):
        self.K, self.P, self.d, self.G, self.h_kv, self.dtype = K, P, d, G, h_kv, dtype
        self.held, self.new, self.cache = list(held), list(new), cache or dtype
        self.softcap, self.window, self.order = softcap, window, order
        rng, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
        lens = [a + b for a, b in zip(held, new)]
        self.lens, self.batch, self.h_q = lens, len(lens), h_kv * G
        self.max_blocks = max(1, max(-(-n // P) for n in lens) + 1)
        self.n_pages = sum(-(-n // P) for n in lens) + spare
        self.tables = C.blocks_of(lens, P, self.max_blocks, self.n_pages, rng, fill=fill)
        kind = C.DT[self.cache]
        self.pools = [C.empty_pool(self.n_pages, P, h_kv, d, order, kind, cuda) for _ in range(2)]
        self.rows = [[torch.randn(n, h_kv, d, generator=g).to(kind) for n in lens] for _ in range(2)]
        for pool, rows in zip(self.pools, self.rows):
            for b, r in enumerate(rows):
                first = max(0, held[b] + 1 - window) if window else 0
                C.put_rows(pool, order, self.tables, P, b, first, r[first:])
        self.tokens = sum(new) + pad
        self.qs = torch.randn(max(1, self.tokens), self.h_q + q_pad, d, generator=g).to(C.DT[dtype]).to(cuda)
        self.q = self.qs[:self.tokens, :self.h_q]
        e4 = self.cache == "e4m3"
        self.scales = [(0.5 + torch.rand(h_kv, generator=g)).to(cuda) if e4 else None for _ in range(2)]
        self.slopes = (2.0 ** -torch.arange(1, self.h_q + 1).float().mul(8 / self.h_q)).to(cuda) if slopes else None
        self.scale = scale or d ** -0.5
        k = C.kinds(K)
        self.desc = K.make_cache_desc(h_q=self.h_q, h_kv=h_kv, head_dim=d, page_size=P, n_pages=self.n_pages, dtype=k[dtype],
                                      cache_dtype=k[self.cache], order=K.ORDER_HEAD if order == "head" else K.ORDER_ROW)
        self.p = K.make_chunk_attend_desc(batch=self.batch, max_blocks=self.max_blocks, max_tokens=self.tokens,
                                          q_stride=(self.h_q + q_pad) * d, scale=scale, softcap=softcap, window=window)
        self.ws = C.workspace(K, K.kvsel_chunk_attend_workspace_size(self.desc, self.p), cuda)
        self.t = torch.from_numpy(self.tables).to(torch.int32).to(cuda)
        self.l = torch.tensor(lens, dtype=torch.int64, device=cuda)
        self.indptr = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int64, device=cuda)
        self.o = torch.full((self.tokens, self.h_q, d), 7.0, dtype=C.DT[dtype], device=cuda)
        self.lse = torch.full((self.tokens, self.h_q), 7.0, device=cuda)

    def run(self, stream=None, lse=True):
        self.K.kvsel_chunk_attend(self.desc, self.p, self.q, self.pools[0], self.pools[1], self.t, self.l, self.indptr, self.slopes,
                                  self.scales[0], self.scales[1], self.o, self.lse if lse else None, self.ws, stream=stream)
        return self

    def check(self, error=None, requests=None, lse=True):
        torch.cuda.synchronize()
        assert self.K.kvsel_read_device_error(self.ws) == (self.K.OK if error is None else error)
        got, ls, q = C.f64(self.o), C.f64(self.lse), C.f64(self.q)
        eps, w = torch.finfo(C.DT[self.dtype]).eps, 2.0 ** -8 if self.cache == "bf16" else 2.0 ** -11
        at = 0
        for b, n in enumerate(self.new):
            x, at = at, at + n
            if requests is not None and b not in requests:
                assert (got[x:at] == 7).all() and (ls[x:at] == 7).all()
                continue
            for h in range(self.h_kv if n else 0):
                hs = slice(h * self.G, (h + 1) * self.G)
                k, v = (C.f64(r[b][:, h]) * (1.0 if s is None else float(s[h])) for r, s in zip(self.rows, self.scales))
                sl = None if self.slopes is None else C.f64(self.slopes)[hs]
                o, l, mass, zmax = O.chunk_attend(q[x:at, hs], k, v, self.held[b], self.scale, self.softcap, self.window, sl)
                rows = min(len(k), self.window or len(k))
                bias = 0.0 if sl is None else float(sl.max()) * rows
                dz = 2 * U * ((self.d + 8) * zmax + 4 * self.softcap + 4 * bias)
                if self.cache == "e4m3":
                    dz += U * self.d * self.scale * np.abs(q[x:at, hs]).max() * np.abs(k).max()
                low = 2 * U * rows * np.abs(v).max() if self.cache != "bf16" else 0.0
                tol = eps / 2 * np.abs(o) + (2 * (dz + 2.0 ** -20 + 2 * U * (rows + 64)) + w) * mass + low
                bad = ~(np.abs(got[x:at, hs] - o) <= tol)
                assert not bad.any(), (b, h, bad.sum(), np.argwhere(bad)[0], got[x:at, hs][bad][0], o[bad][0])
                if lse:
                    bad = ~(np.abs(ls[x:at, hs] - l) <= dz + 2.0 ** -19 * (1 + np.abs(l)) + 2 * U * (rows + 64))
                    assert not bad.any(), (b, h, np.argwhere(bad)[0])
        assert (got[at:] == 7).all() and (ls[at:] == 7).all()           # the padding, as it was
        return self


@pytest.fixture(scope="module")
def K():
    from attention_kv_cache_gb300 import kvsel
    return kvsel


@pytest.mark.parametrize("held,new", [
    ([0], [1]), ([0], [2]), ([127], [1]), ([128], [1]), ([129], [2]), ([0], [129]), ([0], [300]), ([1000], [33]),
    ([0, 5, 700, 0, 31], [40, 0, 9, 1, 64]), ([0, 0], [0, 0]), ([383, 256], [128, 257]), ([4000] * 3 + [0], [1, 2, 3, 0]),
], ids=range(12))
def test_lengths(cuda, K, held, new):
    """From a single token of an empty request to chunks that end inside steps, tiles and pages."""
    Case(K, cuda, held, new).run().check()


@pytest.mark.parametrize("kw", [
    dict(G=1, h_kv=4), dict(G=1, h_kv=1, d=64), dict(G=5), dict(G=7, h_kv=3, d=64), dict(G=8, h_kv=1), dict(G=16, h_kv=2),
    dict(G=40, h_kv=1), dict(G=3, h_kv=2, q_pad=5),
], ids=str)
def test_heads(cuda, K, kw):
    Case(K, cuda, [0, 200, 61], [150, 3, 31], **kw).run().check()


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("order,P,d", [("head", 16, 128), ("row", 24, 64), ("head", 7, 128), ("row", 1, 64), ("head", 64, 64),
                                       ("row", 256, 128), ("head", 100, 128), ("row", 33, 128), ("head", 8, 64)])
def test_pools(cuda, K, dtype, cache, order, P, d):
    """Every pool type over pages that are boxes of 8, 16 and 32 rows, and pages that no box fits."""
    Case(K, cuda, [0, 310, 45], [70, 21, 260], dtype=dtype, cache=cache, order=order, P=P, d=d).run().check()


@pytest.mark.parametrize("kw", [
    dict(softcap=30.0), dict(softcap=0.5), dict(slopes=True), dict(window=1), dict(window=40), dict(window=129, slopes=True),
    dict(window=500), dict(softcap=20.0, slopes=True, window=200), dict(scale=0.3), dict(softcap=2.0, cache="e4m3", window=77),
    dict(slopes=True, cache="e4m3", d=64), dict(window=64, dtype="f16", P=9),
], ids=str)
@pytest.mark.parametrize("new", [[3, 1, 9], [150, 260, 90]], ids=["few", "many"])
def test_masks(cuda, K, kw, new):
    Case(K, cuda, [0, 310, 700], new, **kw).run().check()


def test_work_is_cut_anywhere(cuda, K):
    """More items than CTAs, items of a few steps and one of hundreds: pieces begin and end inside items, tiles in turn."""
    rng = np.random.default_rng(5)
    held = [int(x) for x in rng.integers(0, 900, 40)] + [20000]
    new = [int(x) for x in rng.integers(0, 40, 40)] + [70]
    Case(K, cuda, held, new, G=2, h_kv=8, d=64).run().check()


@pytest.mark.parametrize("G,new", [(4, 5), (4, 20), (4, 50), (1, 100)], ids=["copies", "turns", "two tiles", "tokens"])
@pytest.mark.parametrize("cache", ["bf16", "f16"])
@pytest.mark.parametrize("P", [16, 7])
def test_values_that_are_not_finite_stay_where_they_are_seen(cuda, K, G, new, cache, P):
    """Infinities and NaN in V rows of later tokens, and in rows before a window, reach those that see them alone."""
    held, window = 300, 200
    c = Case(K, cuda, [held], [new], G=G, dtype=cache, P=P, window=window)
    rows = [(held + new // 2, 3, float("inf")), (held + new - 1, 5, float("nan")), (held + 1 - window, 7, float("-inf")),
            (held + 3 - window, 9, float("nan"))]
    for t, col, x in rows:
        v = c.rows[1][0][t:t + 1].clone()
        v[..., col] = x
        C.put_rows(c.pools[1], c.order, c.tables, P, 0, t, v)
    c.run()
    torch.cuda.synchronize()
    got = C.f64(c.o)[:new].copy()
    for t, col, x in rows:
        sees = np.array([t <= held + i and t > held + i - window for i in range(new)])
        assert sees.any() and not sees.all()
        bad = got[sees][..., col]
        assert (np.isnan(bad) if x != x else bad == x).all(), (t, col)
        assert np.isfinite(got[~sees][..., col]).all()
    # the columns that hold none are as they would be, for every token
    plain = Case(K, cuda, [held], [new], G=G, dtype=cache, P=P, window=window).run()
    torch.cuda.synchronize()
    clean = [x for x in range(c.d) if x not in (3, 5, 7, 9)]
    assert torch.equal(c.o[:new][..., clean], plain.o[:new][..., clean]) and torch.equal(c.lse, plain.lse)


def test_long_tail_behind_one_score_is_kept(cuda, K):
    """One score 20 binary orders above 4000 others: their mass is 2^-8 of the row's, each weight 2^-20."""
    for dtype in ("bf16", "f16"):
        c = Case(K, cuda, [4000], [6], G=2, h_kv=1, dtype=dtype, scale=1.0)
        c.q.zero_()
        c.q[..., 0] = 1.0
        for b in range(2):
            c.rows[b][0].zero_()
        c.rows[0][0][17, :, 0] = 20 * np.log(2.0)
        c.rows[1][0][:, :, 1] = 1.0
        c.rows[1][0][17, :, 1] = 0.0
        for i in range(2):
            C.put_rows(c.pools[i], c.order, c.tables, c.P, 0, 0, c.rows[i][0])
        c.run().check()
        assert (c.o[:6, :, 1] > 0.003).all()


@pytest.mark.parametrize("kw", [dict(), dict(dtype="f16"), dict(cache="e4m3"), dict(d=64), dict(slopes=True), dict(softcap=90.0),
                                dict(softcap=500.0, cache="e4m3", dtype="f16")],
                         ids=["bf16", "f16", "e4m3", "heads of 64", "bias", "cap", "far cap"])
@pytest.mark.parametrize("shape", ["rise", "fall", "peaks"])
@pytest.mark.parametrize("new", [[70, 40], [3, 20]], ids=["many", "few"])
def test_scores_that_move_by_a_hundred_binary_orders(cuda, K, kw, shape, new):
    """The largest score so far is passed in every step, in none but the first, or by some keys far above the others."""
    c = Case(K, cuda, [900, 300], new, **kw)
    c.qs[..., 0] = 8.0 * (c.d / 128) ** 0.5
    for b, n in enumerate(c.lens):
        t = torch.arange(n)[:, None]
        ramp = {"rise": t / n, "fall": 1 - t / n, "peaks": (t % 200 == 150).float()}[shape]
        c.rows[0][b][:, :, 0] = (100.0 * ramp).to(c.rows[0][b].dtype)
        C.put_rows(c.pools[0], c.order, c.tables, c.P, b, 0, c.rows[0][b])
    c.run().check()


@pytest.mark.parametrize("cache", ["bf16", "f16", "e4m3"])
def test_rows_begin_where_those_beside_them_rise(cuda, K, cache):
    """Windows that end at a step's edge for some tokens and before it for their neighbours: the step is the first for some rows of a
    warp, and 13 binary orders above the last one for the others.  Requests enough that a CTA has steps in a row."""
    c = Case(K, cuda, [900] * 12, [70] * 12, h_kv=8, dtype="bf16" if cache == "e4m3" else cache, cache=cache, window=163)
    c.qs[..., 0] = 8.0
    for b, n in enumerate(c.lens):
        c.rows[0][b][:, :, 0] = (100.0 * torch.arange(n)[:, None] / n).to(c.rows[0][b].dtype)
        C.put_rows(c.pools[0], c.order, c.tables, c.P, b, 738, c.rows[0][b][738:])
    c.run().check()


@pytest.mark.parametrize("softcap", [0.0, 0.7, 30.0])
@pytest.mark.parametrize("new", [[70, 40], [3, 20]], ids=["many", "few"])
def test_scales_that_are_not_positive(cuda, K, softcap, new):
    c = Case(K, cuda, [900, 300], new, cache="e4m3", softcap=softcap, slopes=softcap == 30.0)
    c.scales[0][0] *= -1
    c.scales[0][1] = 0.0
    c.run().check()


def test_no_lse_and_repeated_calls_agree(cuda, K):
    c = Case(K, cuda, [0, 100, 3000], [200, 1, 40], cache="e4m3").run()
    torch.cuda.synchronize()
    o, lse = c.o.clone(), c.lse.clone()
    c.o.fill_(7), c.lse.fill_(7)
    c.run(lse=False)
    torch.cuda.synchronize()
    assert torch.equal(c.o, o) and (c.lse == 7).all()
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.o, o) and torch.equal(c.lse, lse)


def test_bad_requests_are_left_out(cuda, K):
    """Lengths and offsets out of range: the request is reported and left as it was, the others are right."""
    for what in ("length", "negative", "tokens", "falls"):
        c = Case(K, cuda, [40, 60, 80], [5, 7, 9])
        if what == "length":
            c.l[1] = c.max_blocks * c.P + 1
        elif what == "negative":
            c.l[1] = -1
        elif what == "tokens":
            c.l[1] = 6                                         # fewer rows than new tokens
        if what == "falls":
            c.indptr[3] = c.tokens + 1
            c.run().check(error=K.ERR_INVALID_ARG, requests=[0, 1])
        else:
            c.run().check(error=K.ERR_INVALID_ARG, requests=[0, 2])


@pytest.mark.parametrize("P,cache", [(16, "bf16"), (5, "bf16"), (16, "e4m3"), (5, "e4m3")])
def test_bad_pages_are_left_out(cuda, K, P, cache):
    """A page outside the pool: reported, its rows take no part; a token that sees no other row gives 0 and -inf."""
    c = Case(K, cuda, [300, 0], [4, 3], P=P, cache=cache)
    c.t[0, 2] = c.n_pages
    c.t[1, 0] = -1
    gone = range(2 * P, 3 * P)
    c.run()
    torch.cuda.synchronize()
    assert K.kvsel_read_device_error(c.ws) == K.ERR_DEVICE
    keep = [t for t in range(304) if t not in gone]
    for h in range(c.h_kv):
        hs = slice(h * c.G, (h + 1) * c.G)
        k, v = (C.f64(r[0][:, h]) * (1.0 if s is None else float(s[h])) for r, s in zip(c.rows, c.scales))
        for i in range(4):
            mine = [t for t in keep if t <= 300 + i]
            o = O.paged_attend(C.f64(c.q)[i, hs], k[mine], v[mine], c.scale)[0]
            assert np.abs(C.f64(c.o)[i, hs] - o).max() < 0.02
    assert (c.o[4:7, :, :] == 0).all() == (P >= 3) and torch.isneginf(c.lse[4:7]).all() == (P >= 3)


def test_any_strides(cuda, K):
    """Pools inside a larger one: rows, heads and pages with gaps, pages in an odd order of strides."""
    c = Case(K, cuda, [100, 40], [30, 200], P=16, order="row")
    for i in range(2):
        wide = torch.full((c.h_kv, c.n_pages, c.P, 2 * c.d), float("nan"), dtype=c.pools[i].dtype, device=cuda)
        wide[..., :c.d] = c.pools[i].permute(2, 0, 1, 3)
        c.pools[i] = wide
    c.desc = K.make_cache_desc(h_q=c.h_q, h_kv=c.h_kv, head_dim=c.d, page_size=c.P, n_pages=c.n_pages, dtype=K.DTYPE_BF16,
                               strides=(c.P * 2 * c.d, c.n_pages * c.P * 2 * c.d, 2 * c.d))
    c.run().check()


def test_offsets_past_32_bits(cuda, K):
    """Pages more than 2^31 elements from the pool's start."""
    c = Case(K, cuda, [200], [20], h_kv=1, G=2)
    far = 2 ** 22                                               # pages 2^22 apart in a pool of 2^31 elements and more
    n = c.P * c.d
    stride = (2 ** 31 // (c.n_pages - 1) // n + 1) * n
    for i in range(2):
        big = torch.empty((c.n_pages - 1) * stride + n, dtype=c.pools[i].dtype, device=cuda)
        big.as_strided((c.n_pages, n), (stride, 1)).copy_(c.pools[i].view(c.n_pages, n))
        c.pools[i] = big
    assert far and (c.n_pages - 1) * stride >= 2 ** 31
    c.desc = K.make_cache_desc(h_q=c.h_q, h_kv=1, head_dim=c.d, page_size=c.P, n_pages=c.n_pages, dtype=K.DTYPE_BF16,
                               strides=(stride, n, c.d))
    c.run().check()


def test_streams_and_capture(cuda, K):
    """On a side stream, and captured: a replay reads lengths, offsets and tables as they are then."""
    c = Case(K, cuda, [100, 500, 33], [40, 1, 8], pad=20)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.run(stream=side)
    side.synchronize()
    c.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    c.o.fill_(7), c.lse.fill_(7)
    graph.replay()
    c.check()
    # another split of the same rows into held and new ones
    c.held, c.new = [139, 480, 1], [1, 21, 40]
    c.indptr.copy_(torch.tensor([0, 1, 22, 62]))
    c.o.fill_(7), c.lse.fill_(7)
    graph.replay()
    c.check()


def test_a_prompt_by_chunks_is_the_prompt_at_once(cuda, K):
    whole = Case(K, cuda, [0], [600], seed=4, pad=0)
    whole.run()
    torch.cuda.synchronize()
    for first, n in ((0, 250), (250, 1), (251, 349)):
        part = Case(K, cuda, [first], [n], pad=0, seed=4)
        part.rows = [[r[0][:first + n]] for r in whole.rows]
        for i in range(2):
            C.put_rows(part.pools[i], part.order, part.tables, part.P, 0, 0, part.rows[i][0])
        part.q.copy_(whole.q[first:first + n])
        part.run().check()
        assert (part.lse - whole.lse[first:first + n]).abs().max() < 1e-5
