"""The paged calls at the ends of their descriptors' ranges."""

import numpy as np
import pytest
import torch

from oracle import paged_oracle as O
from tests import paged_common as C
from tests.test_gpu_paged_attend import Case

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("lens", [[0, 1, 40, 700], [5000]])
def test_the_largest_and_the_smallest_cap(cuda, cache, dtype, lens):
    """A cap of 2^127 leaves every score as it is, one of 2^-126 makes all of them zero."""
    from attention_kv_cache_gb300 import kvsel as K
    c = Case(K, cuda, lens, cache=cache, dtype=dtype, softcap=2.0 ** 127, seed=4).run()
    c.softcap = 0.0                                      # the definition, and the tolerance, of no cap
    c.check()
    c = Case(K, cuda, lens, cache=cache, dtype=dtype, softcap=2.0 ** -126, seed=4).run()
    c.softcap, c.scale = 0.0, 0.0
    c.check()
    c = Case(K, cuda, lens, cache=cache, dtype=dtype, softcap=2.0 ** -126, seed=4)
    c.q.zero_()
    c.run()
    c.softcap = 0.0
    c.check()


@pytest.mark.parametrize("P,blocks,short", [(8, 2 ** 28 - 2, 0), (8, 2 ** 28 - 2, 5), (1, 2 ** 31 - 2, 0), (20, 107374181, 0)])
@pytest.mark.parametrize("window", [40, 40000])
def test_the_longest_request_that_a_table_describes(cuda, P, blocks, short, window):
    """Lengths up to 2^31 - 2, of which a window is seen: by one CTA, and by all lanes."""
    from attention_kv_cache_gb300 import kvsel as K
    h_q, h_kv, d, n_pages = 4, 2, 128, 50
    n = blocks * P - short
    assert (blocks + 1) * P < 2 ** 31 and blocks * P > 2 ** 31 - 32
    g = torch.Generator().manual_seed(P)
    pools = [torch.randn(n_pages, h_kv, P, d, generator=g).bfloat16() for _ in range(2)]
    q = torch.randn(1, h_q, d, generator=g).bfloat16()
    slopes = 2.0 ** -torch.arange(4.0, 4.0 + h_q) / 8
    t = torch.arange(n - window, n)
    pages = torch.randint(0, n_pages, (int(t[-1]) // P - int(t[0]) // P + 1,), generator=g)
    table = torch.full((1, blocks), -7, dtype=torch.int32, device=cuda)              # what is not seen is not looked up
    table[0, int(t[0]) // P:int(t[-1]) // P + 1] = pages.to(torch.int32).to(cuda)
    desc = K.make_cache_desc(h_q=h_q, h_kv=h_kv, head_dim=d, page_size=P, n_pages=n_pages)
    p = K.make_paged_attend_desc(batch=1, max_blocks=blocks, window=window)
    ws = C.workspace(K, K.kvsel_paged_attend_workspace_size(desc, p), cuda)
    o, lse = torch.full((1, h_q, d), 7.0, dtype=torch.bfloat16, device=cuda), torch.full((1, h_q), 7.0, device=cuda)
    K.kvsel_paged_attend(desc, p, q.to(cuda), pools[0].to(cuda), pools[1].to(cuda), table,
                         torch.tensor([n], device=cuda), slopes.to(cuda), None, None, o, lse, ws)
    torch.cuda.synchronize()
    assert K.kvsel_read_device_error(ws) == K.OK
    at = pages[t // P - int(t[0]) // P]
    k, v = (C.f64(x)[at.numpy(), :, (t % P).numpy()] for x in pools)                  # [window, h_kv, d]
    for h in range(h_kv):
        hs = slice(h * 2, h * 2 + 2)
        sl = C.f64(slopes)[hs]
        want, ls, mass, zmax = O.paged_attend(C.f64(q)[0, hs], k[:, h], v[:, h], d ** -0.5, 0.0, 0, sl)
        dz = 2 * U * ((d + 8) * zmax + 4 * sl.max() * window)
        tol = 2.0 ** -8 * np.abs(want) + 2 * (dz + 2.0 ** -17 + 2 * U * (window + 64)) * mass
        assert (np.abs(C.f64(o)[0, hs] - want) <= tol).all()
        assert (np.abs(C.f64(lse)[0, hs] - ls) <= dz + 2.0 ** -20 * (1 + np.abs(ls)) + 2 * U * (window + 64)).all()


def test_the_longest_request_is_assigned(cuda):
    """The last rows that a table describes: in place, and out of place."""
    from attention_kv_cache_gb300 import kvsel as K
    P, blocks = 8, 2 ** 28 - 2
    n = blocks * P - 11
    i64 = dict(dtype=torch.int64, device=cuda)
    table = torch.full((1, blocks), 5, dtype=torch.int32, device=cuda)
    ws = C.workspace(K, K.kvsel_page_assign_workspace_size(1), cuda)
    for in_place in (False, True):
        lens, head = torch.tensor([n], **i64), torch.zeros(1, **i64)
        lens_out, head_out = (lens, head) if in_place else (torch.empty(1, **i64), torch.empty(1, **i64))
        slots, pos, ids = torch.empty(12, **i64), torch.empty(12, **i64), torch.empty(12, dtype=torch.int32, device=cuda)
        K.kvsel_page_assign(P, 9, lens, torch.tensor([11], **i64), torch.tensor([7, 2], dtype=torch.int32, device=cuda), head, table,
                            lens_out, head_out, torch.empty(2, **i64), slots, pos, ids, ws)
        torch.cuda.synchronize()
        assert K.kvsel_read_device_error(ws) == K.OK
        assert lens_out.tolist() == [n + 11] and head_out.tolist() == [1] and table[0, -2:].tolist() == [5, 7]
        rows = list(range(n, n + 11))
        assert slots.tolist() == [(7 if t // P == blocks - 1 else 5) * P + t % P for t in rows] + [-1]
        assert pos.tolist() == rows + [0] and ids.tolist() == [0] * 11 + [-1]
        lens.fill_(n + 1)                                # one row too many: nothing is assigned
        K.kvsel_page_assign(P, 9, lens, torch.tensor([11], **i64), torch.tensor([7, 2], dtype=torch.int32, device=cuda), head, table,
                            lens_out, head_out, torch.empty(2, **i64), slots, pos, ids, ws)
        torch.cuda.synchronize()
        assert K.kvsel_read_device_error(ws) == K.ERR_INVALID_ARG and slots.tolist() == [-1] * 12


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_capped_scores_over_every_argument(cuda, sign):
    """The lse of one row is its capped score: every bf16 argument from 2^-7 to 16, across the change of form at 1/4.

    tanh is off by 2^-20 of itself below 1/4 and by 2^-21 above; three fp32 roundings follow (the cap in base 2, the product
    with it and with ln 2)."""
    from attention_kv_cache_gb300 import kvsel as K
    x = torch.cat([(1 + torch.arange(128).float() / 128) * 2.0 ** e for e in range(-7, 4)]) * sign
    h_q, d, P = 16, 128, 16
    q = torch.zeros(len(x) // h_q, h_q, d)
    q[:, :, 0] = x.reshape(-1, h_q)
    k = torch.zeros(1, 1, P, d)
    k[..., 0] = 1.0
    for cap in (1.0, 8.0):                               # (a power of two: the scores are exact multiples of it)
        qd, kd = (q * cap).bfloat16().to(cuda), k.bfloat16().to(cuda)
        desc = K.make_cache_desc(h_q=h_q, h_kv=1, head_dim=d, page_size=P, n_pages=1)
        p = K.make_paged_attend_desc(batch=len(q), max_blocks=1, scale=1.0, softcap=cap)
        ws = C.workspace(K, K.kvsel_paged_attend_workspace_size(desc, p), cuda)
        o, lse = torch.empty(len(q), h_q, d, dtype=torch.bfloat16, device=cuda), torch.empty(len(q), h_q, device=cuda)
        K.kvsel_paged_attend(desc, p, qd, kd, kd, torch.zeros(len(q), 1, dtype=torch.int32, device=cuda),
                             torch.ones(len(q), dtype=torch.int64, device=cuda), None, None, None, o, lse, ws)
        torch.cuda.synchronize()
        got, want = C.f64(lse).reshape(-1) / cap, np.tanh(C.f64(x))
        tol = np.where(np.abs(C.f64(x)) < 0.25, 2.0 ** -20 * np.abs(want), 2.0 ** -21) + 3 * U * np.abs(want)
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (x[bad][:5], (np.abs(got - want) / tol).max())
