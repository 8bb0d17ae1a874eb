"""One-token attention over a paged pool against the fp64 definition.

Every row that a request does not see is NaN in the pool: rows behind its end and before its window, spare
pages, and the entries of its table behind its last page are outside the pool.

Tolerances (u = 2^-24, fp32 rounding).  A score is off by at most
    dz = 2 u ((d + 8) zmax + 4 |cap| + 4 bias) (+ u d scale max|q| max|k| where the query row is held in fp16),
zmax the largest scale sum_c |q_c k_c|, bias the largest |slope (t - (n - 1))| (products exact, up to d truncating
additions, a few roundings of the score).  A weight is then off by exp(dz), 2^-22 of ex2 and 2^-18 of the two-part P
(2^-9 of a 2^-9 remainder), and sums of n terms by 2 u (n + 64).  With mass = sum p |v| / sum p,
    |o - ref| <= eps/2 |ref| + 2 (dz + 2^-17 + 2 u (n + 64)) mass (+ 2 u n max|v|: fp16 weights below its normal range),
eps/2 the rounding to the output's type, and |lse - ref| <= dz + 2^-20 (1 + |ref|) + 2 u (n + 64).
"""

import numpy as np
import pytest
import torch

from oracle import paged_oracle as O
from tests import paged_common as C

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


class Case:
    """Inputs of one call, and its outputs' references."""

    def __init__(self, K, cuda, lens, h_kv=2, G=4, d=128, P=16, dtype="bf16", cache=None, order="head", softcap=0.0,
                 window=0, slopes=False, scale=0.0, seed=0, spare=3, max_blocks=None, q_pad=0, qmul=1.0):
        self.K, self.lens, self.P, self.d, self.G, self.h_kv, self.dtype = K, list(lens), P, d, G, h_kv, dtype
        self.cache = cache or dtype
        self.order, self.softcap, self.window = order, softcap, window
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        batch, h_q = len(lens), h_kv * G
        self.batch, self.h_q = batch, h_q
        self.max_blocks = max_blocks or max(1, max(-(-n // P) for n in lens) + 1)
        self.n_pages = sum(-(-n // P) for n in lens) + spare
        self.tables = C.blocks_of(lens, P, self.max_blocks, self.n_pages, rng)
        kind = C.DT[self.cache]
        self.pools = [C.empty_pool(self.n_pages, P, h_kv, d, order, kind, cuda) for _ in range(2)]
        self.rows = [[torch.randn(n, h_kv, d, generator=g).to(kind) for n in lens] for _ in range(2)]
        for pool, rows in zip(self.pools, self.rows):
            for b, r in enumerate(rows):
                first = max(0, lens[b] - window) if window else 0
                C.put_rows(pool, order, self.tables, P, b, first, r[first:])
        self.qs = torch.randn(batch, h_q + q_pad, d, generator=g).mul(qmul).to(C.DT[dtype]).to(cuda)
        self.q = self.qs[:, :h_q]
        e4 = self.cache == "e4m3"
        self.scales = [(0.5 + torch.rand(h_kv, generator=g)).to(cuda) if e4 else None for _ in range(2)]
        self.slopes = (2.0 ** -torch.arange(1, h_q + 1).float().mul(8 / h_q)).to(cuda) if slopes else None
        self.scale = scale or d ** -0.5
        k = C.kinds(K)
        self.desc = K.make_cache_desc(h_q=h_q, h_kv=h_kv, head_dim=d, page_size=P, n_pages=self.n_pages, dtype=k[dtype],
                                      cache_dtype=k[self.cache], order=K.ORDER_HEAD if order == "head" else K.ORDER_ROW)
        self.p = K.make_paged_attend_desc(batch=batch, max_blocks=self.max_blocks, q_stride=(h_q + q_pad) * d,
                                          softcap=softcap, window=window, scale=scale)
        self.ws = C.workspace(K, K.kvsel_paged_attend_workspace_size(self.desc, self.p), cuda)
        self.t = torch.from_numpy(self.tables).to(torch.int32).to(cuda)
        self.l = torch.tensor(lens, dtype=torch.int64, device=cuda)
        self.o = torch.full((batch, h_q, d), 7.0, dtype=C.DT[dtype], device=cuda)
        self.lse = torch.full((batch, h_q), 7.0, device=cuda)

    def run(self, stream=None):
        self.K.kvsel_paged_attend(self.desc, self.p, self.q, self.pools[0], self.pools[1], self.t, self.l, self.slopes,
                                  self.scales[0], self.scales[1], self.o, self.lse, self.ws, stream=stream)
        return self

    def check(self, lens=None, error=None, keep=None):
        torch.cuda.synchronize()
        assert self.K.kvsel_read_device_error(self.ws) == (self.K.OK if error is None else error)
        got, lse, q = C.f64(self.o), C.f64(self.lse), C.f64(self.q)
        eps = torch.finfo(C.DT[self.dtype]).eps
        for b, n in enumerate(self.lens if lens is None else lens):
            for h in range(self.h_kv):
                hs = slice(h * self.G, (h + 1) * self.G)
                k, v = (C.f64(r[b][:n, h]) * (1.0 if s is None else float(s[h]))
                        for r, s in zip(self.rows, self.scales))
                if keep is not None:
                    k, v = k[keep(b)], v[keep(b)]
                sl = None if self.slopes is None else C.f64(self.slopes)[hs]
                o, ls, mass, zmax = O.paged_attend(q[b, hs], k, v, self.scale, self.softcap, self.window, sl)
                if n == 0 or len(k) == 0:
                    assert (got[b, hs] == 0).all() and np.isneginf(lse[b, hs]).all()
                    continue
                bias = 0.0 if sl is None else float(sl.max()) * min(n, self.window or n)
                dz = 2 * U * ((self.d + 8) * zmax + 4 * self.softcap + 4 * bias)
                if self.cache == "e4m3":
                    dz += U * self.d * self.scale * np.abs(q[b, hs]).max() * np.abs(k).max()
                low = 2 * U * n * np.abs(v).max() if "bf16" not in (self.cache,) else 0.0
                tol = eps / 2 * np.abs(o) + 2 * (dz + 2.0 ** -17 + 2 * U * (n + 64)) * mass + low
                bad = ~(np.abs(got[b, hs] - o) <= tol)
                assert not bad.any(), (b, h, bad.sum(), np.argwhere(bad)[0], got[b, hs][bad][0], o[bad][0])
                tl = dz + 2.0 ** -20 * (1 + np.abs(ls)) + 2 * U * (n + 64)
                assert (np.abs(lse[b, hs] - ls) <= tl).all(), (b, h, lse[b, hs], ls)


LENS = [0, 1, 31, 32, 33, 500]

SHAPES = [
    dict(lens=LENS),
    dict(lens=LENS, order="row", dtype="f16"),
    dict(lens=LENS, cache="e4m3"),
    dict(lens=LENS, cache="e4m3", dtype="f16", order="row", d=64),
    dict(lens=LENS, d=64, G=1, h_kv=3),
    dict(lens=LENS, d=64, dtype="f16", G=5, h_kv=1, P=64),
    dict(lens=LENS, G=8, P=256),
    dict(lens=LENS, G=8, P=48, order="row"),
    dict(lens=LENS, G=16, h_kv=1, P=32),
    dict(lens=LENS, G=16, cache="e4m3", h_kv=1, P=32),
    dict(lens=LENS, G=12, d=64, dtype="f16"),
    dict(lens=LENS, G=20, h_kv=1, dtype="bf16"),                   # two tiles of query heads, the second partly empty
    dict(lens=LENS, G=40, h_kv=1, d=64, cache="e4m3"),
    dict(lens=LENS, P=1),
    dict(lens=LENS, P=7, cache="e4m3"),
    dict(lens=LENS, P=20, order="row"),
    dict(lens=LENS, P=17, d=64, dtype="f16"),
    dict(lens=LENS, P=255, cache="e4m3", d=64),
    dict(lens=[1]),
    dict(lens=[20000], seed=5),                                    # one request over every lane
    dict(lens=[9000, 0, 3, 12345], G=8, order="row", seed=6),
    dict(lens=[5001], h_kv=1, G=2, d=64, cache="e4m3", P=16),
    dict(lens=[64] * 40 + [0] + [2000], h_kv=8, G=1, P=16),       # more requests than some lanes
    dict(lens=list(range(0, 200)), h_kv=5, G=2, d=64),             # more requests than lanes
    dict(lens=list(range(1, 300)), h_kv=8, G=16, d=64, P=32, dtype="f16"),
    dict(lens=[40, 0, 70], h_kv=1300, G=1, d=64),                  # more KV heads than warps
    dict(lens=[i % 37 for i in range(4096)], h_kv=1, G=2, d=64, P=8),
    dict(lens=[i % 5 for i in range(4095)] + [700], h_kv=1, G=1, P=16, cache="e4m3"),
]


@pytest.mark.parametrize("kw", SHAPES, ids=lambda k: "-".join(f"{a}{b if not isinstance(b, list) else len(b)}" for a, b in k.items()))
def test_shapes(cuda, kw):
    from attention_kv_cache_gb300 import kvsel as K
    Case(K, cuda, **kw).run().check()


@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("kw", [
    dict(softcap=5.0), dict(softcap=50.0, qmul=8.0), dict(slopes=True), dict(window=1), dict(window=33),
    dict(window=64, slopes=True, softcap=20.0), dict(window=100000), dict(scale=1.0), dict(q_pad=3), dict(qmul=60.0),
    dict(window=250, P=20), dict(softcap=1e6),
], ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()))
def test_options(cuda, kw, cache, dtype):
    """Capped scores, distance biases, sliding windows, other scales, strided queries, peaked softmaxes."""
    from attention_kv_cache_gb300 import kvsel as K
    Case(K, cuda, [0, 1, 40, 700, 2049], cache=cache, dtype=dtype, seed=9, **kw).run().check()


@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("kw", [
    dict(), dict(G=16), dict(G=1, d=64, h_kv=3), dict(G=20, h_kv=1), dict(softcap=9.0, slopes=True), dict(window=40),
    dict(P=7), dict(order="row", q_pad=2), dict(lens=[1]), dict(lens=[0, 0]), dict(lens=[3] * 70, h_kv=2, G=2, d=64),
    dict(qmul=50.0), dict(lens=[64, 380], G=9, P=32), dict(lens=[4000, 4001, 4031, 4032, 4033, 31, 32], window=33),
    dict(lens=[3000 + 7 * i for i in range(14)], window=64, h_kv=2), dict(lens=[2500, 2530], window=1),
], ids=lambda k: "-".join(f"{a}{b if not isinstance(b, list) else len(b)}" for a, b in k.items()) or "plain")
def test_short_calls(cuda, kw, cache, dtype):
    """Tables that hold few rows: a CTA per request and KV head, no join."""
    from attention_kv_cache_gb300 import kvsel as K
    before = K.kvsel_launch_count()
    c = Case(K, cuda, **{**dict(lens=[0, 1, 33, 129, 380], cache=cache, dtype=dtype, seed=21), **kw}).run()
    assert K.kvsel_launch_count() == before + 1
    c.check()
    bad = Case(K, cuda, [100, 50, 70], cache=cache, dtype=dtype)
    bad.l[1] = -3
    bad.t[2, 1] = bad.n_pages
    gone = set(range(16, 32))
    torch.cuda.synchronize()
    bad.run()
    torch.cuda.synchronize()
    assert K.kvsel_read_device_error(bad.ws) in (K.ERR_INVALID_ARG, K.ERR_DEVICE)
    bad.check(lens=[100, 0, 70], keep=lambda b: [t for t in range((100, 0, 70)[b]) if b < 2 or t not in gone])


def test_bf16_queries_of_any_size_over_an_8_bit_pool(cuda):
    """The fp16 copy of a bf16 query row is scaled by its own power of two."""
    from attention_kv_cache_gb300 import kvsel as K
    for mul, scale in ((1e20, 1e-20), (1e-20, 1e20), (1e5, 1e-6)):
        Case(K, cuda, [100, 33], cache="e4m3", qmul=mul, scale=scale).run().check()
    c = Case(K, cuda, [100, 33], cache="e4m3")
    c.q.zero_()
    c.run().check()


def test_infinities_and_nan_in_seen_rows_follow_the_softmax(cuda):
    from attention_kv_cache_gb300 import kvsel as K
    c = Case(K, cuda, [40, 3000, 64])
    c.pools[0].nan_to_num_(0.0)
    page = int(c.tables[1, 100])
    c.pools[0][page, 0, 3, 5] = float("nan")          # one key of request 1, KV head 0
    c.run()
    torch.cuda.synchronize()
    assert torch.isnan(c.o[1, :4]).all() and torch.isnan(c.lse[1, :4]).all()
    assert torch.isfinite(c.o[1, 4:].float()).all() and torch.isfinite(c.o[[0, 2]].float()).all()
    c = Case(K, cuda, [40, 3000, 64])                  # every key of a request
    c.pools[0].fill_(float("nan"))
    c.run()
    torch.cuda.synchronize()
    assert torch.isnan(c.o.float()).all()


def test_bad_lengths_and_pages_are_reported(cuda):
    from attention_kv_cache_gb300 import kvsel as K
    c = Case(K, cuda, [100, 50, 70])
    for bad in (-1, c.max_blocks * c.P + 1, 2 ** 40):
        c.l.copy_(torch.tensor([100, bad, 70]))
        c.run().check(lens=[100, 0, 70], error=K.ERR_INVALID_ARG)
    c.l.copy_(torch.tensor([100, 50, 70]))
    for bad in (-1, "the pool's size", 2 ** 31 - 1, -2 ** 31):
        for P in (16, 7):                              # pages of whole boxes of rows, and others
            c = Case(K, cuda, [100, 50, 70], P=P)
            c.t[0, 2] = c.n_pages if bad == "the pool's size" else bad
            gone = set(range(2 * P, 3 * P))
            c.run().check(error=K.ERR_DEVICE, keep=lambda b: [t for t in range(c.lens[b]) if b or t not in gone])
    c = Case(K, cuda, [10, 50])
    c.t[0, 0] = -5                                      # nothing left
    c.run().check(error=K.ERR_DEVICE, keep=lambda b: [] if b == 0 else list(range(50)))


def test_rows_past_32_bit_offsets(cuda):
    """A pool of more than 2^32 bytes and 2^31 elements, its pages far apart."""
    from attention_kv_cache_gb300 import kvsel as K
    c = Case(K, cuda, [60, 33], h_kv=1, G=4, spare=0)
    n, P, d = c.n_pages, c.P, c.d
    stride = (2 ** 31 // (n - 1) + 128) // 8 * 8 + 8
    big = torch.empty((n - 1) * stride + 2 * P * d, dtype=torch.bfloat16, device=cuda)
    k, v = (torch.as_strided(big, (n, 1, P, d), (stride, P * d, d, 1), off) for off in (0, P * d))
    k.copy_(c.pools[0])
    v.copy_(c.pools[1])
    assert k.stride(0) * (n - 1) > 2 ** 31
    c.desc.page_stride, c.desc.head_stride = stride, P * d
    c.pools = [k, v]
    c.run().check()


def test_packed_cache_through_strides(cuda):
    """A packed [h_kv][rows][d] cache read as pages of 16 rows."""
    from attention_kv_cache_gb300 import kvsel as K
    h_kv, rows, d, P = 2, 160, 128, 16
    c = Case(K, cuda, [150], h_kv=h_kv)
    packed = [torch.zeros(h_kv, rows, d, dtype=torch.bfloat16, device=cuda) for _ in range(2)]
    for p, r in zip(packed, c.rows):
        p[:, :150] = r[0].transpose(0, 1).to(cuda)
    c.desc = K.make_cache_desc(h_q=8, h_kv=h_kv, head_dim=d, page_size=P, n_pages=rows // P,
                               strides=(P * d, rows * d, d))
    c.pools = packed
    c.t.copy_(torch.arange(c.max_blocks, dtype=torch.int32))
    c.run().check()


def test_same_bits_every_time_and_workspace_shared(cuda):
    """Two calls, and calls of other shapes on the same workspace between them, give the same bits."""
    from attention_kv_cache_gb300 import kvsel as K
    a = Case(K, cuda, [700, 9000, 3], G=8, seed=1)
    b = Case(K, cuda, [5, 4000], G=16, h_kv=1, seed=2)
    n = max(a.ws.numel(), b.ws.numel())
    a.ws = b.ws = C.workspace(K, n, cuda)
    a.run()
    first = a.o.clone(), a.lse.clone()
    for _ in range(3):
        b.run()
        a.o.zero_()
        a.run()
        torch.cuda.synchronize()
        assert torch.equal(a.o.view(torch.int16), first[0].view(torch.int16)) and torch.equal(a.lse, first[1])
    a.check()
    b.check()


def test_two_streams_at_once_and_graph_replay(cuda):
    from attention_kv_cache_gb300 import kvsel as K
    cases = [Case(K, cuda, [3000, 100], seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(cases, streams):
            c.run(stream=s)
    for c in cases:
        c.check()
    c = cases[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    want = c.o.clone()
    c.o.zero_()
    g.replay()
    c.check()
    assert torch.equal(c.o, want)
    c.l.copy_(torch.tensor([17, 0]))                     # a replay reads the lengths of its time
    g.replay()
    c.check(lens=[17, 0])


def test_no_lse_wanted(cuda):
    from attention_kv_cache_gb300 import kvsel as K
    c = Case(K, cuda, [0, 9000, 40])
    c.run()
    want, ls = c.o.clone(), c.lse
    c.o.zero_()
    c.lse = None
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.o, want)
    c.lse = ls
    c.check()


@pytest.mark.parametrize("seed", range(16))
def test_random_shapes(cuda, seed):
    from attention_kv_cache_gb300 import kvsel as K
    r = np.random.default_rng(1000 + seed)
    dtype = str(r.choice(["bf16", "f16"]))
    n = int(r.integers(1, 7))
    Case(K, cuda, [int(x) for x in r.integers(0, int(r.choice([40, 600, 5000])), n)], h_kv=int(r.choice([1, 2, 3, 8])),
         G=int(r.choice([1, 3, 4, 8, 9, 16, 17])), d=int(r.choice([64, 128])), P=int(r.choice([8, 16, 32, 64, r.integers(1, 257)])),
         dtype=dtype, cache=str(r.choice([dtype, "e4m3"])), order=str(r.choice(["head", "row"])),
         softcap=float(r.choice([0, 0, 15.0])), window=int(r.choice([0, 0, r.integers(1, 3000)])),
         slopes=bool(r.random() < 0.3), seed=seed).run().check()
