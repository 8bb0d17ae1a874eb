"""Arguments of the calls for prompt chunks, shared prefixes and beams that are refused on the host, and their definitions
against independent ones (no GPU)."""

import ctypes
import math

import numpy as np
import pytest
import torch

from attention_kv_cache_gb300 import kvsel as K
from oracle import paged_oracle as O

BIG = 1 << 40


def _raw(name, *args):
    return K.raw_call(name, *args)


def _cache(**kw):
    base = dict(h_q=8, h_kv=2, head_dim=128, page_size=16, n_pages=10)
    base.update(kw)
    return K.make_cache_desc(**base)


# ------------------------------------------------------------------------------------------- chunks
@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), K.ERR_INVALID_ARG), (dict(batch=4097), K.ERR_INVALID_ARG), (dict(max_blocks=0), K.ERR_INVALID_ARG),
    (dict(max_blocks=2 ** 27), K.ERR_INVALID_ARG), (dict(max_tokens=-1), K.ERR_INVALID_ARG),
    (dict(max_tokens=2 ** 31), K.ERR_INVALID_ARG), (dict(max_tokens=2 ** 30), K.ERR_UNSUPPORTED),
    (dict(max_tokens=2 ** 28, max_blocks=2 ** 20), K.ERR_UNSUPPORTED),
    (dict(q_stride=-8), K.ERR_INVALID_ARG), (dict(q_stride=1028), K.ERR_INVALID_ARG), (dict(scale=-1.0), K.ERR_INVALID_ARG),
    (dict(scale=math.nan), K.ERR_INVALID_ARG), (dict(softcap=-1.0), K.ERR_INVALID_ARG), (dict(softcap=1e-40), K.ERR_INVALID_ARG),
    (dict(window=-1), K.ERR_INVALID_ARG),
])
def test_bad_chunk_descriptor(kw, status):
    p = K.make_chunk_attend_desc(**{**dict(batch=2, max_blocks=4, max_tokens=64), **kw})
    n = ctypes.c_size_t(0)
    assert _raw("kvsel_chunk_attend_workspace_size", _cache(), p, ctypes.byref(n)) == status
    assert _raw("kvsel_chunk_attend", _cache(), p, 16, 16, 32, 16, 16, 16, None, None, None, 48, None, 256, BIG, None) == status


@pytest.mark.parametrize("call", ["chunk", "prefix"])
def test_rows_heads_and_pointers(call):
    n = ctypes.c_size_t(0)
    chunk = K.make_chunk_attend_desc(batch=2, max_blocks=4, max_tokens=64)
    step = K.make_paged_attend_desc(batch=2, max_blocks=4)

    def run(c=None, q=16, k=16, v=32, table=16, lens=16, a=16, b=16, slopes=None, ks=None, vs=None, o=48, lse=None, ws=256):
        if call == "chunk":
            return _raw("kvsel_chunk_attend", c or _cache(), chunk, q, k, v, table, lens, a, slopes, ks, vs, o, lse, ws, BIG, None)
        return _raw("kvsel_prefix_attend", c or _cache(), step, 1, q, k, v, table, lens, a, b, slopes, ks, vs, o, lse, ws, BIG,
                    None)
    for d in (16, 96, 256):
        if call == "chunk":
            assert _raw("kvsel_chunk_attend_workspace_size", _cache(head_dim=d), chunk, ctypes.byref(n)) == K.ERR_UNSUPPORTED
        assert run(c=_cache(head_dim=d)) == K.ERR_UNSUPPORTED
    bad = [dict(q=None), dict(k=None), dict(v=None), dict(table=None), dict(lens=None), dict(a=None), dict(o=None), dict(q=8),
           dict(k=8), dict(v=24), dict(o=8), dict(lens=4), dict(a=4), dict(table=2), dict(slopes=2), dict(lse=2), dict(o=16),
           dict(ks=16, vs=16), dict(ks=16), dict(c=_cache(cache_dtype=K.DTYPE_E4M3)),
           dict(c=_cache(cache_dtype=K.DTYPE_E4M3), vs=16)]
    if call == "prefix":
        bad += [dict(b=None), dict(b=4)]
    for kw in bad:
        assert run(**kw) == K.ERR_INVALID_ARG, kw
    assert run(ws=None) == K.ERR_WORKSPACE
    assert run(ws=128) == K.ERR_WORKSPACE


def test_chunk_of_no_tokens_does_nothing():
    p = K.make_chunk_attend_desc(batch=2, max_blocks=4, max_tokens=0)
    assert _raw("kvsel_chunk_attend", _cache(), p, None, None, None, None, None, None, None, None, None, None, None, None, 0,
                None) == K.OK


@pytest.mark.parametrize("groups", [0, -1, 3])
def test_bad_groups(groups):
    step = K.make_paged_attend_desc(batch=2, max_blocks=4)
    n = ctypes.c_size_t(0)
    assert _raw("kvsel_prefix_attend_workspace_size", _cache(), step, groups, ctypes.byref(n)) == K.ERR_INVALID_ARG
    assert _raw("kvsel_prefix_attend", _cache(), step, groups, 16, 16, 32, 16, 16, 16, 16, None, None, None, 48, None, 256, BIG,
                None) == K.ERR_INVALID_ARG


# -------------------------------------------------------------------------------------------- beams
@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), K.ERR_INVALID_ARG), (dict(beams=0), K.ERR_INVALID_ARG), (dict(n_out=0), K.ERR_INVALID_ARG),
    (dict(vocab=0), K.ERR_INVALID_ARG), (dict(dtype=K.DTYPE_E4M3), K.ERR_INVALID_ARG), (dict(pad_token=-1), K.ERR_INVALID_ARG),
    (dict(pad_token=1000), K.ERR_INVALID_ARG), (dict(beams=1, vocab=5, n_out=6), K.ERR_INVALID_ARG),
    (dict(row_stride=-1), K.ERR_INVALID_ARG), (dict(beams=65), K.ERR_UNSUPPORTED), (dict(n_out=65), K.ERR_UNSUPPORTED),
    (dict(batch=2000), K.ERR_UNSUPPORTED), (dict(beams=64, vocab=8192 * 129), K.ERR_UNSUPPORTED),
])
def test_bad_select_descriptor(kw, status):
    p = K.make_beam_select_desc(**{**dict(batch=2, beams=4, n_out=8, vocab=1000), **kw})
    n = ctypes.c_size_t(0)
    assert _raw("kvsel_beam_select_workspace_size", ctypes.byref(p), ctypes.byref(n)) == status
    assert _raw("kvsel_beam_select", p, 16, 16, None, 32, 48, 64, None, 256, BIG, None) == status


def test_select_pointers():
    p = K.make_beam_select_desc(batch=2, beams=4, n_out=8, vocab=1000)
    assert K.kvsel_beam_select_workspace_size(p) % K.WS_ALIGN == 0

    def run(x=16, s=16, e=None, so=32, pa=48, t=64, lse=None, ws=256, nb=BIG):
        return _raw("kvsel_beam_select", p, x, s, e, so, pa, t, lse, ws, nb, None)
    for kw in (dict(x=None), dict(s=None), dict(so=None), dict(pa=None), dict(t=None), dict(x=17), dict(s=18), dict(so=34),
               dict(pa=50), dict(t=66), dict(lse=2), dict(so=16)):
        assert run(**kw) == K.ERR_INVALID_ARG, kw
    for kw in (dict(ws=None), dict(ws=128), dict(nb=256)):
        assert run(**kw) == K.ERR_WORKSPACE, kw


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), K.ERR_INVALID_ARG), (dict(beams=0), K.ERR_INVALID_ARG), (dict(max_blocks=0), K.ERR_INVALID_ARG),
    (dict(n_layers=0), K.ERR_INVALID_ARG), (dict(layer_stride=-8), K.ERR_INVALID_ARG), (dict(beams=65), K.ERR_UNSUPPORTED),
    (dict(batch=2049), K.ERR_UNSUPPORTED), (dict(batch=2048, max_blocks=2 ** 20), K.ERR_UNSUPPORTED),
])
def test_bad_reorder_descriptor(kw, status):
    p = K.make_beam_reorder_desc(**{**dict(batch=2, beams=2, max_blocks=8, n_layers=2, layer_stride=1024), **kw})
    n = ctypes.c_size_t(0)
    assert _raw("kvsel_beam_reorder_workspace_size", ctypes.byref(p), ctypes.byref(n)) == status
    assert _raw("kvsel_beam_reorder", _cache(), p, 16, 16, 16, 16, 4, 16, 16, 16, 16, 32, 48, 256, BIG, None) == status


def test_reorder_pointers():
    def run(c=None, pa=16, l=16, t=16, f=16, n=4, h=16, to=16, lo=16, ho=16, k=32, v=48, ws=256, nb=BIG, **kw):
        p = K.make_beam_reorder_desc(**{**dict(batch=2, beams=2, max_blocks=8, n_layers=2, layer_stride=1024), **kw})
        return _raw("kvsel_beam_reorder", c or _cache(), p, pa, l, t, f, n, h, to, lo, ho, k, v, ws, nb, None)
    for kw in (dict(pa=None), dict(l=None), dict(t=None), dict(f=None), dict(h=None), dict(to=None), dict(lo=None), dict(ho=None),
               dict(k=None), dict(v=None), dict(k=48), dict(k=40), dict(v=40), dict(l=20), dict(h=20), dict(lo=20), dict(ho=20),
               dict(pa=18), dict(t=18), dict(f=18), dict(to=18), dict(n=-1), dict(n=2 ** 31), dict(layer_stride=1028),
               dict(max_blocks=2 ** 27, batch=1, beams=1)):
        assert run(**kw) == K.ERR_INVALID_ARG, kw
    for kw in (dict(ws=None), dict(ws=128), dict(nb=256)):
        assert run(**kw) == K.ERR_WORKSPACE, kw


# ------------------------------------------------------------------------------------- definitions
def test_chunk_definition_is_the_attention_of_torch():
    g = torch.Generator().manual_seed(1)
    n, first, G, d = 5, 7, 3, 16
    q, k, v = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((n, G, d), (first + n, d), (first + n, d)))
    o, lse, mass, _ = O.chunk_attend(q.numpy(), k.numpy(), v.numpy(), first, d ** -0.5)
    mask = torch.arange(first + n) <= first + torch.arange(n)[:, None]
    ref = torch.nn.functional.scaled_dot_product_attention(q.transpose(0, 1), k.expand(G, -1, -1), v.expand(G, -1, -1), attn_mask=mask)
    assert np.allclose(o, ref.transpose(0, 1).numpy(), atol=1e-12)
    z = (q.transpose(0, 1) @ k.T * d ** -0.5).masked_fill(~mask, -math.inf)
    assert np.allclose(lse, torch.logsumexp(z, -1).T.numpy(), atol=1e-12) and (mass >= np.abs(o) - 1e-12).all()


def test_select_definition_by_enumeration():
    rng = np.random.default_rng(2)
    x, s = rng.normal(size=(3, 7)), np.array([-1.0, -0.5, -np.inf])
    scores, parents, tokens, lse = O.beam_select(x, s, 10, ended=[0, 1, 0], pad_token=4)
    assert np.allclose(lse, torch.logsumexp(torch.from_numpy(x), -1).numpy())
    z = s[:, None] + torch.log_softmax(torch.from_numpy(x), -1).numpy()
    z[1] = -np.inf
    z[1, 4] = -0.5
    order = np.argsort(-z.reshape(-1), kind="stable")[:10]
    assert (parents * 7 + tokens == order).all() and np.allclose(scores, z.reshape(-1)[order], rtol=1e-14)


def test_reorder_definition_keeps_every_page_once():
    """A step of page ownership by hand: pages shared by two beams, a dead beam, twins with a part-full last page."""
    tables = [[0, 1, 2, 9], [0, 1, 3, 9], [0, 4, 5, 9]]
    out = O.beam_reorder(4, [[0, 0, 1]], [10, 10, 12], tables, [-1] * 6 + [7, 8], 6)
    t, lens, queue, head, copies = out
    # beam 2's pages 4 and 5 are freed, in front of the queue's head; the twin of beam 0 takes page 4 for its copy of page 2
    assert queue.tolist() == [-1, -1, -1, -1, 4, 5, 7, 8] and head == 5
    assert t.tolist() == [[0, 1, 2, 9], [0, 1, 4, 9], [0, 1, 3, 9]] and lens.tolist() == [10, 10, 10]
    assert copies == [(1, 2, 2, 4, 2)]
    assert O.beam_reorder(4, [[0, 0, 0]], [10, 0, 0], tables, [-1] * 6 + [7], 6) is None
