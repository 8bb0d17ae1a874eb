"""Norm, rotation and the write of new rows into a paged pool, against the fp64 definition.

Tolerances (u = 2^-24).  With a norm the mean square of d values is off by (16 + log2 d) u relative, its root's
reciprocal by half of that and 2 u of rsqrtf, the scaled value by 3 u more: under 2^-19 relative.  cos and sin are
off by 2^-32 of a turn, the rounding of the angle to fp32 (at most pi u < 2^-22) and the fast functions' 2^-21:
under 2^-20; a turned value is two such products.  With size = factor (|a| + |b|) of
its pair, |y - ref| <= 2^-18 size before the rounding to the output's type, which adds eps / 2 |y| (and half a step
of the type's smallest numbers).  Values that pass unturned without a norm, and the v rows of a 16-bit pool, are
exact.
"""

import numpy as np
import pytest
import torch

from oracle import paged_oracle as O
from tests import paged_common as C

pytestmark = pytest.mark.gpu
# half a step relative to the value, eps / 2: 8, 11 and 4 significant bits (1.0750706 lies between the bf16 neighbours
# 1.0703125 and 1.078125, 2^-7 apart, and rounds to the second, off by 0.0030544 <= 2^-8 * 1.0750706 = 0.0041995)
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "e4m3": 2.0 ** -4}
SMALLEST = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "e4m3": 2.0 ** -10}
SENTINEL = 3.0


def near(got, want, size, kind, what):
    want = np.clip(want, -O.E4M3_MAX, O.E4M3_MAX) if kind == "e4m3" else want
    delta = 2.0 ** -18 * size
    tol = HALF_STEP[kind] * (np.abs(want) + delta) + delta + SMALLEST[kind]
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, bad.sum(), np.argwhere(bad)[0], got[bad][0], want[bad][0])


class Case:
    def __init__(self, K, cuda, n, h_q=8, h_kv=2, d=128, P=16, dtype="bf16", cache=None, order="head", norm=True, rot=None,
                 layout="half", scaling="plain", pos_max=131072, bias=0.0, pad=0, seed=0, fused=True, mul=1.0):
        self.K, self.n, self.dtype, self.cache, self.order, self.P = K, n, dtype, cache or dtype, order, P
        self.layout, self.bias, self.h_q, self.h_kv, self.d = layout, bias, h_q, h_kv, d
        rng, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
        t = C.DT[dtype]
        x = torch.randn(n, h_q + 2 * h_kv, d, generator=g).mul(mul).to(t).to(cuda)
        self.q, self.k, self.v = x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:]
        if not fused:                                   # heads outside tokens
            self.q, self.k, self.v = (y.transpose(0, 1).contiguous().transpose(0, 1) for y in (self.q, self.k, self.v))
        self.n_pages = -(-n // P) + 4
        slots = rng.permutation(self.n_pages * P)[:n].astype(np.int64)
        if pad:
            slots[rng.permutation(n)[:pad]] = -1
        self.slots_h, self.pos_h = slots, rng.integers(0, pos_max, n)
        self.slots, self.pos = torch.from_numpy(slots).to(cuda), torch.from_numpy(self.pos_h).to(cuda)
        self.rot = d if rot is None else rot
        self.freq, self.factor = O.rope_freqs(self.rot, scaling, 10000.0, 8.0) if self.rot else (None, 1.0)
        self.freq_d = None if self.freq is None else torch.from_numpy(self.freq).to(cuda)
        self.w = [(1 + 0.2 * torch.randn(d, generator=g)).to(t).to(cuda) if norm else None for _ in range(2)]
        e4 = self.cache == "e4m3"
        self.scales = [(0.02 + 0.02 * torch.rand(h_kv, generator=g)).to(cuda) if e4 else None for _ in range(2)]
        self.pools = []
        for _ in range(2):
            p = C.empty_pool(self.n_pages, P, h_kv, d, order, C.DT[self.cache], cuda, nan=False)
            p.copy_(torch.full(p.shape, SENTINEL))
            self.pools.append(p)
        self.q_out = torch.full((n, h_q, d), SENTINEL, dtype=t, device=cuda)
        kk = C.kinds(K)
        self.desc = K.make_cache_desc(h_q=h_q, h_kv=h_kv, head_dim=d, page_size=P, n_pages=self.n_pages, dtype=kk[dtype],
                                      cache_dtype=kk[self.cache], order=K.ORDER_HEAD if order == "head" else K.ORDER_ROW)
        self.rope = K.make_rope_desc(rot_dim=self.rot, layout=K.ROPE_HALF if layout == "half" else K.ROPE_INTERLEAVED,
                                     factor=self.factor, norm_eps=1e-6, weight_bias=bias, q=self.q, k=self.k, v=self.v)
        self.ws = C.workspace(K, K.WS_ALIGN, cuda)
        self.in_h = [C.f64(y) for y in (self.q, self.k, self.v)]

    def run(self, stream=None, **kw):
        a = dict(q=self.q, k=self.k, v=self.v, q_out=self.q_out, kc=self.pools[0], vc=self.pools[1], slots=self.slots)
        a.update(kw)
        has_kv = a["k"] is not None
        self.K.kvsel_rope_append(self.desc, self.rope, a["q"], a["k"], a["v"], self.pos, a["slots"], self.w[0],
                                 self.w[1], self.freq_d, a["q_out"], a["kc"], a["vc"],
                                 self.scales[0] if has_kv else None, self.scales[1] if has_kv else None, self.ws,
                                 stream=stream)
        return self

    def turned(self, x, w):
        return O.norm_rope(x, self.pos_h, self.freq, float(np.float32(self.factor)), self.layout,
                           None if w is None else C.f64(w), self.bias, 1e-6)

    def check(self, error=None, q=True, kv=True):
        torch.cuda.synchronize()
        assert self.K.kvsel_read_device_error(self.ws) == (self.K.OK if error is None else error)
        total = self.n_pages * self.P
        real = self.slots_h != -1
        got = C.f64(self.q_out)
        if q:
            y, size = self.turned(self.in_h[0], self.w[0])
            near(got[real], y[real], size[real], self.dtype, "q")
            assert (got[~real] == SENTINEL).all()
        else:
            assert (got == SENTINEL).all()
        stored = real & (self.slots_h >= 0) & (self.slots_h < total) & kv
        s = self.slots_h[stored]
        for i, (pool, x, w, scale) in enumerate(zip(self.pools, self.in_h[1:], (self.w[1], None), self.scales)):
            p = C.f64(C.pool_view(pool, self.order)).reshape(total, self.h_kv, self.d)
            y, size = self.turned(x, w) if i == 0 else (x, np.abs(x))
            y, size = y[stored], size[stored]
            if scale is not None:
                f = C.f64(scale)[:, None]
                y, size = y / f, size / f
            if i == 1 and scale is None:
                assert (p[s] == y).all()
            else:
                near(p[s], y, size, self.cache, "kv"[i])
            rest = np.ones(total, bool)
            rest[s] = False
            assert (p[rest] == SENTINEL).all()


@pytest.mark.parametrize("kw", [
    dict(n=1), dict(n=1, h_q=1, h_kv=1, d=16, P=1, rot=16), dict(n=7, pad=3), dict(n=300, pad=40, P=7),
    dict(n=33, dtype="f16", order="row", layout="interleaved"), dict(n=33, layout="interleaved", rot=32),
    dict(n=33, rot=32, scaling="banded"), dict(n=33, rot=0), dict(n=33, norm=False), dict(n=33, norm=False, rot=0),
    dict(n=65, cache="e4m3", scaling="ramp"), dict(n=65, cache="e4m3", dtype="f16", order="row", P=20, mul=30.0),
    dict(n=20, d=64, h_q=3, h_kv=3, scaling="linear"), dict(n=20, d=80, rot=80), dict(n=20, d=96, rot=48, dtype="f16"),
    dict(n=20, d=112, layout="interleaved"), dict(n=20, d=256, cache="e4m3"), dict(n=20, d=256, layout="interleaved"),
    dict(n=20, d=32, h_q=33, h_kv=11), dict(n=40, fused=False), dict(n=40, bias=1.0), dict(n=50, pos_max=2 ** 31),
    dict(n=3000, h_q=32, h_kv=8), dict(n=5, h_q=600, h_kv=300), dict(n=700, h_q=1, h_kv=1, pad=99),
    dict(n=100, h_q=5, h_kv=1, cache="e4m3", d=48, rot=48), dict(n=3001, h_q=16, h_kv=1, d=64, dtype="f16", layout="interleaved", rot=16),
], ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()))
def test_rows(cuda, kw):
    from attention_kv_cache_gb300 import kvsel as K
    Case(K, cuda, **kw).run().check()


def test_broadcast_heads_and_tokens(cuda):
    """Strides of zero: one row for every head, one token's rows for every token."""
    from attention_kv_cache_gb300 import kvsel as K
    c = Case(K, cuda, 50, h_q=4, h_kv=4)
    c.k = c.k[:, :1].expand(-1, 4, -1)
    c.v = c.v[:1].expand(50, -1, -1)
    c.rope.k_head_stride, c.rope.v_stride = c.k.stride(1), c.v.stride(0)
    assert c.rope.k_head_stride == 0 and c.rope.v_stride == 0
    c.in_h[1:] = [C.f64(c.k), C.f64(c.v)]
    c.run().check()


def test_far_positions_lose_nothing(cuda):
    """At 2^31 positions a 32-bit angle would be off by a turn and more; the pairs of frequency 1 keep 2^-18."""
    from attention_kv_cache_gb300 import kvsel as K
    c = Case(K, cuda, 64, norm=False, dtype="f16")
    c.pos_h[:] = np.arange(64) * 33554393 % (2 ** 31)
    c.pos_h[-1] = 2 ** 31 - 1
    c.pos.copy_(torch.from_numpy(c.pos_h))
    c.run().check()


def test_queries_or_rows_alone_and_in_place(cuda):
    from attention_kv_cache_gb300 import kvsel as K
    c = Case(K, cuda, 19, pad=2)
    c.run(k=None, v=None, kc=None, vc=None).check(kv=False)
    c = Case(K, cuda, 19)
    c.run(k=None, v=None, kc=None, vc=None, slots=None).check(kv=False)
    c = Case(K, cuda, 19, pad=2)
    c.run(q=None, q_out=None).check(q=False)
    c = Case(K, cuda, 19)
    own = c.q.contiguous()
    c.rope.q_stride, c.rope.q_head_stride = own.stride(0), own.stride(1)
    c.run(q=own, q_out=own)
    c.q_out = own
    c.check()


def test_slots_outside_the_pool_are_reported_and_not_written(cuda):
    from attention_kv_cache_gb300 import kvsel as K
    for bad in (-2, None, 2 ** 40, -2 ** 62):
        c = Case(K, cuda, 9)
        c.slots_h[4] = c.n_pages * c.P if bad is None else bad
        c.slots.copy_(torch.from_numpy(c.slots_h))
        c.run().check(error=K.ERR_DEVICE)


def test_values_past_the_8_bit_range_clamp_and_nan_stays(cuda):
    from attention_kv_cache_gb300 import kvsel as K
    c = Case(K, cuda, 4, cache="e4m3", norm=False, rot=0, dtype="bf16")
    c.v[0, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 1e30], device=cuda)
    c.run()
    torch.cuda.synchronize()
    s = int(c.slots_h[0])
    row = C.pool_view(c.pools[1], c.order)[s // c.P, s % c.P, 0, :4].float().cpu().tolist()
    assert row[0] == 448 and row[1] == -448 and row[2] != row[2] and row[3] == 448


def test_another_stream_and_a_captured_call(cuda):
    from attention_kv_cache_gb300 import kvsel as K
    c = Case(K, cuda, 100, pad=3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(stream=s).check()
    c = Case(K, cuda, 100, pad=3)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        c.run()
    g.replay()
    c.check()


def test_pool_offsets_past_32_bits(cuda):
    from attention_kv_cache_gb300 import kvsel as K
    c = Case(K, cuda, 40, h_kv=1)
    n, P, d = c.n_pages, c.P, c.d
    stride = (2 ** 31 // (n - 1) + 128) // 8 * 8 + 8
    big = torch.empty((n - 1) * stride + 2 * P * d, dtype=torch.bfloat16, device=cuda)
    pools = [torch.as_strided(big, (n, 1, P, d), (stride, P * d, d, 1), off) for off in (0, P * d)]
    for p in pools:
        p.fill_(SENTINEL)
    c.pools = pools
    c.desc.page_stride, c.desc.head_stride = stride, P * d
    c.run().check()
