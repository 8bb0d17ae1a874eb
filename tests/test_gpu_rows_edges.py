"""Attention of many rows at the ends of its range."""

import numpy as np
import pytest
import torch

from oracle import paged_oracle as O
from tests import paged_common as C
from tests.test_gpu_chunk_attend import Case as Chunk
from tests.test_gpu_prefix_attend import Case as Prefix

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def K():
    from attention_kv_cache_gb300 import kvsel
    return kvsel


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new", [[40, 70], [3, 5]], ids=["many", "few"])
@pytest.mark.parametrize("k_scale", [1e-16, 1e-37, 1e-44])
def test_scales_of_almost_nothing(cuda, K, dtype, new, k_scale):
    """8-bit keys of a scale that leaves nothing of a score, and queries of zeros: the mean of the rows that are seen."""
    c = Chunk(K, cuda, [300, 77], new, dtype=dtype, cache="e4m3")
    c.scales[0].fill_(k_scale)
    c.q[::2].zero_()
    c.run().check()


@pytest.mark.parametrize("k_scale", [1e-16, 1e-37])
def test_scales_of_almost_nothing_behind_a_prefix(cuda, K, k_scale):
    c = Prefix(K, cuda, [(400, [1, 200, 30]), (150, [3] * 40)], cache="e4m3", window=300)
    c.scales[0].fill_(k_scale)
    c.q[::2].zero_()
    c.run().check()


@pytest.mark.parametrize("P,blocks,short", [(8, 2 ** 28 - 2, 0), (8, 2 ** 28 - 2, 5), (1, 2 ** 31 - 2, 0), (16, 2 ** 27 - 2, 3), (20, 107374181, 0)])
@pytest.mark.parametrize("window,new", [(40, 5), (4000, 90)])
def test_the_longest_request_behind_a_window(cuda, K, P, blocks, short, window, new):
    """Lengths up to 2^31 - 2, of which windows are seen; rows behind the last are NaN."""
    h_q, h_kv, d, n_pages = 4, 2, 128, 50
    n = blocks * P - short
    g = torch.Generator().manual_seed(P)
    pools = [torch.randn(n_pages, h_kv, P, d, generator=g).bfloat16() for _ in range(2)]
    q = torch.randn(new, h_q, d, generator=g).bfloat16()
    slopes = 2.0 ** -torch.arange(4.0, 4.0 + h_q) / 8
    t = torch.arange(n - new + 1 - window, n)
    first = int(t[0]) // P
    pages = torch.randint(0, n_pages - 1, (int(t[-1]) // P - first + 1,), generator=g)
    pages[-1] = n_pages - 1                                                           # (of the last page's rows alone)
    if n % P:
        for x in pools:
            x[n_pages - 1, :, n % P:] = float("nan")
    table = torch.full((1, blocks), -7, dtype=torch.int32, device=cuda)
    table[0, first:first + len(pages)] = pages.to(torch.int32).to(cuda)
    desc = K.make_cache_desc(h_q=h_q, h_kv=h_kv, head_dim=d, page_size=P, n_pages=n_pages)
    p = K.make_chunk_attend_desc(batch=1, max_blocks=blocks, max_tokens=new, window=window)
    ws = C.workspace(K, K.kvsel_chunk_attend_workspace_size(desc, p), cuda)
    o, lse = torch.full((new, h_q, d), 7.0, dtype=torch.bfloat16, device=cuda), torch.full((new, h_q), 7.0, device=cuda)
    K.kvsel_chunk_attend(desc, p, q.to(cuda), pools[0].to(cuda), pools[1].to(cuda), table, torch.tensor([n], device=cuda),
                         torch.tensor([0, new], device=cuda), slopes.to(cuda), None, None, o, lse, ws)
    torch.cuda.synchronize()
    assert K.kvsel_read_device_error(ws) == K.OK
    at = pages[t // P - first]
    k, v = (C.f64(x)[at.numpy(), :, (t % P).numpy()] for x in pools)                  # [rows, h_kv, d]
    for h in range(h_kv):
        hs = slice(h * 2, h * 2 + 2)
        sl = C.f64(slopes)[hs]
        # (the first token's window ends `new - 1` rows before the last one's: rows are numbered from the first that is seen)
        want, ls, mass, zmax = O.chunk_attend(C.f64(q)[:, hs], k[:, h], v[:, h], len(t) - new, d ** -0.5, 0.0, window, sl)
        dz = 2 * U * ((d + 8) * zmax + 4 * sl.max() * window)
        tol = 2.0 ** -8 * np.abs(want) + (2 * (dz + 2.0 ** -20 + 2 * U * (window + 64)) + 2.0 ** -8) * mass
        assert (np.abs(C.f64(o)[:, hs] - want) <= tol).all()
        assert (np.abs(C.f64(lse)[:, hs] - ls) <= dz + 2.0 ** -19 * (1 + np.abs(ls)) + 2 * U * (window + 64)).all()


def every_row(pools, q, n, P, period, blocks, scale, pos):
    """fp64 (o, lse, mass) of q [h_q, d] over rows 0 .. pos of n, whose pages repeat every `period`; one KV head."""
    k, v = (C.f64(x)[:, 0].reshape(-1, x.shape[-1]) for x in pools)                   # rows of the pages
    z = C.f64(q) @ k.T * scale
    m = z.max(-1, keepdims=True)
    w = np.exp(z - m)                                                                 # [h_q, period * P]
    count = np.array([(blocks - 1 - c) // period + 1 for c in range(period)], np.float64).repeat(P)
    behind = np.arange(pos + 1, blocks * P) % (period * P)
    np.subtract.at(count, behind, 1.0)
    w = w * count
    total = w.sum(-1, keepdims=True)
    return w @ v / total, (m + np.log(total))[:, 0], w @ np.abs(v) / total


@pytest.mark.parametrize("call,new", [("chunk", 3), ("chunk", 70), ("prefix", 0)])
@pytest.mark.parametrize("P", [8, 16])
def test_all_rows_of_the_longest_request(cuda, K, call, new, P):
    """2^24 steps of 128 keys, seen by every token: what is read of a step's place and count stays below 2^31.

    The kernel's CTAs add some 2^24 / 150 steps each, in fp32: a sum by one addition a step and an output by eight, each off by a
    step of the last place (2^-23) at most."""
    blocks, period, d, h_q = 2 ** 31 // P - 2, 50, 64, 2
    n, g = blocks * P, torch.Generator().manual_seed(P + new)
    pools = [torch.randn(period, 1, P, d, generator=g).bfloat16() for _ in range(2)]
    pools[1] += 4
    desc = K.make_cache_desc(h_q=h_q, h_kv=1, head_dim=d, page_size=P, n_pages=period)
    table = (torch.arange(blocks, dtype=torch.int32, device=cuda) % period).repeat(1 if call == "chunk" else 2, 1)
    k, v = (x.to(cuda) for x in pools)
    steps = 2 ** 24 / torch.cuda.get_device_properties(cuda).multi_processor_count + 2
    if call == "chunk":
        p = K.make_chunk_attend_desc(batch=1, max_blocks=blocks, max_tokens=new)
        ws = C.workspace(K, K.kvsel_chunk_attend_workspace_size(desc, p), cuda)
        rows = list(range(n - new, n))
    else:
        p = K.make_paged_attend_desc(batch=2, max_blocks=blocks)
        ws = C.workspace(K, K.kvsel_prefix_attend_workspace_size(desc, p, 1), cuda)
        rows = [n - 1, n - P // 2]
    q = torch.randn(len(rows), h_q, d, generator=g).bfloat16()
    o, lse = torch.full((len(rows), h_q, d), 7.0, dtype=torch.bfloat16, device=cuda), torch.full((len(rows), h_q), 7.0, device=cuda)
    i64 = dict(dtype=torch.int64, device=cuda)
    if call == "chunk":
        K.kvsel_chunk_attend(desc, p, q.to(cuda), k, v, table, torch.tensor([n], **i64), torch.tensor([0, new], **i64), None, None, None,
                             o, lse, ws)
    else:
        K.kvsel_prefix_attend(desc, p, q.to(cuda), k, v, table, torch.tensor([x + 1 for x in rows], **i64), torch.tensor([0, 2], **i64),
                              torch.tensor([n - P], **i64), None, None, None, o, lse, ws)
    torch.cuda.synchronize()
    assert K.kvsel_read_device_error(ws) == K.OK
    for i, pos in enumerate(rows):
        want, ls, mass = every_row(pools, q[i], n, P, period, blocks, d ** -0.5, pos)
        assert (np.abs(C.f64(lse)[i] - ls) <= 2.0 ** -23 * steps + 2.0 ** -16).all()
        assert (np.abs(C.f64(o)[i] - want) <= 2.0 ** -8 * np.abs(want) + (9 * 2.0 ** -23 * steps + 2.0 ** -8 + 2.0 ** -16) * mass).all()


def test_offsets_that_fall(cuda, K):
    """The request whose offsets fall is reported and left out; the one behind it has the tokens that its own offsets say."""
    c = Chunk(K, cuda, [40, 60, 80], [0, 7, 9])
    c.indptr.copy_(torch.tensor([7, 7, 0, 9]))
    c.new = [0, 0, 9]
    c.run().check(error=K.ERR_INVALID_ARG)
