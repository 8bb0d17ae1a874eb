"""Attention over a long tail of small weights behind a few large ones, against sums in 64 bits.

Every score is a product of small powers and integers, so keys repeat page by page: a table names one page many times,
and the definition sums each page's rows once with its count.

Tolerances (u = 2^-24).  With dz = 2 u (d + 8) zmax for a score, 2^-22 of ex2, 2^-18 of P's two 16-bit parts and 2 u (n + 64) for
a sum of n terms, as for any softmax, o is off by at most
    eps/2 |o| + 2 (dz + 2^-17 + 2 u (n + 64)) mass + n 2^-38 max|v|,    mass = sum p |v| / sum p:
a part in fp16 is a multiple of 2^-24 and the largest weight is held between 2^13 and 2^15, so a weight is off by at most 2^-25 / 2^13 of
the largest (nothing of the kind in bf16).  Half a step of the output's smallest numbers is added.  The tail carries `mass`, so
a tail that is dropped, or counted in the sum of the weights alone, is far outside.
"""

import math

import numpy as np
import pytest
import torch

from tests import paged_common as C

pytestmark = pytest.mark.gpu
U, P, D = 2.0 ** -24, 16, 128
KINDS = [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")]


def attend(cuda, cache, dtype, pages, levels, v, batch=1, G=4):
    """One request, `batch` times: its table lists `pages`; every row of page i has the score levels[i] (natural
    logarithms) but for row 0 of page 0, whose score is levels[-1]; v [pages, P, D].  Returns (o, lse) and their references."""
    from attention_kv_cache_gb300 import kvsel as K
    kind, n_pages = C.DT[cache], len(levels) - 1
    k = torch.zeros(n_pages, 1, P, D)
    for i in range(n_pages):
        k[i, 0, :, 0] = levels[i]
    k[0, 0, 0, 0] = levels[-1]
    k, v = k.to(kind), v[:, None].to(kind)
    assert C.f64(k[0, 0, 0, 0]) == levels[-1] and all(C.f64(k[i, 0, 1, 0]) == levels[i] for i in range(n_pages))
    q = torch.zeros(batch, G, D)
    q[:, :, 0] = 1.0
    n = len(pages) * P
    kk, e4 = C.kinds(K), cache == "e4m3"
    desc = K.make_cache_desc(h_q=G, h_kv=1, head_dim=D, page_size=P, n_pages=n_pages, dtype=kk[dtype], cache_dtype=kk[cache])
    p = K.make_paged_attend_desc(batch=batch, max_blocks=len(pages), scale=1.0)
    ws = C.workspace(K, K.kvsel_paged_attend_workspace_size(desc, p), cuda)
    one = torch.ones(1, device=cuda) if e4 else None
    o = torch.full((batch, G, D), 7.0, dtype=C.DT[dtype], device=cuda)
    lse = torch.full((batch, G), 7.0, device=cuda)
    table = torch.tensor(pages, dtype=torch.int32, device=cuda).expand(batch, -1).contiguous()
    K.kvsel_paged_attend(desc, p, q.to(C.DT[dtype]).to(cuda), k.to(cuda), v.to(cuda), table,
                         torch.full((batch,), n, dtype=torch.int64, device=cuda), None, one, one, o, lse, ws)
    torch.cuda.synchronize()
    assert K.kvsel_read_device_error(ws) == K.OK
    zs, vs = C.f64(k[:, 0, :, 0]), C.f64(v[:, 0])
    count = np.bincount(pages, minlength=n_pages).astype(float)
    w = np.exp(zs - zs.max()) * count[:, None]
    ref = (w[..., None] * vs).sum((0, 1)) / w.sum()
    mass = (w[..., None] * np.abs(vs)).sum((0, 1)) / w.sum()
    dz = 2 * U * (D + 8) * np.abs(zs).max()
    rel = dz + 2.0 ** -17 + 2 * U * (n + 64)
    fp16 = dtype == "f16"
    tol = torch.finfo(C.DT[dtype]).eps / 2 * np.abs(ref) + 2 * rel * mass + (2.0 ** -25 if fp16 else 0.0)
    if cache != "bf16":
        tol = tol + n * 2.0 ** -38 * np.abs(vs).max()
    lref = zs.max() + math.log(w.sum())
    return C.f64(o), C.f64(lse), ref, tol, lref, dz + 2.0 ** -20 * (1 + abs(lref)) + 2 * U * (n + 64)


def check(got, lse, ref, tol, lref, ltol):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (bad.sum(), np.abs(got - ref).max(), ref[:3], tol[:3])
    assert (np.abs(lse - lref) <= ltol).all(), (lse, lref)


def tail(n_pages, low, seed=0):
    """Values of one sign; those of page 0's first row (the high score's) are zero."""
    g = torch.Generator().manual_seed(seed)
    v = low + torch.rand(n_pages, P, D, generator=g)
    v[0, 0] = 0.0
    return v


# scores of the high row and of the rest: 24.2, 25.2, 28.9 and 34.6 binary orders between them
GAPS = [(18.0, 1.25), (18.0, 0.5), (20.0, 0.0), (24.0, 0.0)]


@pytest.mark.parametrize("cache,dtype", KINDS)
@pytest.mark.parametrize("high,low", GAPS)
@pytest.mark.parametrize("rows,batch,at", [(131072, 1, 0), (131072, 1, 4000), (40000, 3, 2499), (16384, 600, 3), (1024, 1, 0), (1024, 2, 63),
                                           (48, 300, 1)])
def test_a_long_tail_behind_one_high_score(cuda, cache, dtype, high, low, rows, batch, at):
    """Requests over many lanes, in one CTA, and more requests than lanes; the high score's page first, inside and last."""
    pages = [1] * (rows // P)
    pages[at] = 0
    check(*attend(cuda, cache, dtype, pages, [low, low, high], tail(2, 0.5), batch=batch))


@pytest.mark.parametrize("cache,dtype", KINDS)
@pytest.mark.parametrize("rise", [0.5, 1.0, 2.0, 4.0, 8.0, 16.0])
def test_scores_that_rise_page_by_page(cuda, cache, dtype, rise):
    """Levels that pass the largest score so far by less and by more than what moves the offset, each held for three steps."""
    levels = [rise * i for i in range(8)]
    pages = [i for i in range(8) for _ in range(6)]
    g = torch.Generator().manual_seed(3)
    check(*attend(cuda, cache, dtype, pages, levels + [0.0], torch.randn(8, P, D, generator=g)))
    check(*attend(cuda, cache, dtype, pages * 60, levels + [0.0], torch.randn(8, P, D, generator=g)))


@pytest.mark.parametrize("cache,dtype", KINDS)
def test_scores_that_fall_page_by_page(cuda, cache, dtype):
    levels = [28.0, 24.0, 20.0, 16.0, 12.0, 8.0, 4.0, 0.0]
    pages = [0] + [1] * 7 + [2] * 80 + [3] * 400 + [4] * 900 + [5] * 1500 + [6] * 3000 + [7] * 9000
    v = tail(8, 0.5, seed=4)
    check(*attend(cuda, cache, dtype, pages, levels + [28.0], v))


@pytest.mark.parametrize("cache,dtype", KINDS)
def test_the_lse_of_one_page_of_equal_rows(cuda, cache, dtype):
    for z in (0.0, 0.125, -0.25, 3.0, -24.0, 256.0):
        o, lse, ref, tol, *_ = attend(cuda, cache, dtype, [0], [z, z], torch.ones(1, P, D))
        want = z + math.log(P)
        assert (np.abs(lse - want) <= 2.0 ** -20 * (1 + abs(want))).all(), (z, lse)
        assert (np.abs(o - ref) <= tol).all()


@pytest.mark.parametrize("rows_before", [64, 1000, 20000])
def test_values_at_the_types_largest(cuda, rows_before):
    """A weight is at most one whatever the offset was taken from: a value near bf16's largest stays finite under a later,
    higher score (5 above the rows before it, whose weights e^-5 have values of zero)."""
    pages = [1] * (rows_before // P) + [0]
    v = torch.zeros(2, P, D)
    v[0, 0] = torch.linspace(1e38, 3.3e38, D)
    v[0, 0, 1::2] *= -1
    check(*attend(cuda, "bf16", "bf16", pages, [0.0, 0.0, 5.0], v))
    check(*attend(cuda, "bf16", "bf16", pages, [0.0, 0.0, 5.0], v, batch=300))
