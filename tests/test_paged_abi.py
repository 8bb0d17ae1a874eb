"""The paged calls refuse bad arguments on the host (no GPU), and their fp64 definitions against other ones."""

import ctypes
import math

import numpy as np
import pytest
import torch

from attention_kv_cache_gb300 import kvsel as K
from oracle import paged_oracle as O

BIG = 1 << 40


def _cache(**kw):
    base = dict(h_q=8, h_kv=2, head_dim=128, page_size=16, n_pages=100)
    base.update(kw)
    return K.make_cache_desc(**base)


def _raw(name, *args):
    return K.raw_call(name, *[ctypes.byref(a) if isinstance(a, ctypes.Structure) else a for a in args])


BAD_CACHES = [
    (dict(h_q=6, h_kv=4), K.ERR_INVALID_ARG),
    (dict(h_kv=0), K.ERR_INVALID_ARG),
    (dict(page_size=0), K.ERR_INVALID_ARG),
    (dict(page_size=257), K.ERR_INVALID_ARG),
    (dict(n_pages=0), K.ERR_INVALID_ARG),
    (dict(n_pages=2 ** 31), K.ERR_INVALID_ARG),
    (dict(dtype=K.DTYPE_E4M3), K.ERR_INVALID_ARG),
    (dict(dtype=3), K.ERR_INVALID_ARG),
    (dict(cache_dtype=K.DTYPE_F16), K.ERR_INVALID_ARG),          # a pool of the other 16-bit type
    (dict(head_dim=0), K.ERR_INVALID_ARG),
    (dict(head_dim=72), K.ERR_UNSUPPORTED),
    (dict(head_dim=272), K.ERR_UNSUPPORTED),
    (dict(strides=(4096, 2048, 132)), K.ERR_INVALID_ARG),        # rows off the 16-byte grid
    (dict(strides=(4096, -2048, 128)), K.ERR_INVALID_ARG),
    (dict(cache_dtype=K.DTYPE_E4M3, strides=(4096, 2048, 136)), K.ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_pool_refused_by_every_call(kw, status):
    c = _cache(**kw)
    n = ctypes.c_size_t(0)
    p = K.make_paged_attend_desc(batch=2, max_blocks=4)
    assert _raw("kvsel_paged_attend_workspace_size", c, p, ctypes.byref(n)) == status
    assert _raw("kvsel_paged_attend", c, p, 16, 16, 32, 16, 16, None, None, None, 16, None, 256, BIG, None) == status
    r = K.make_rope_desc(rot_dim=0)
    assert _raw("kvsel_rope_append", c, r, 4, 16, 16, 16, None, 16, None, None, None, 16, 16, 32, None, None, None,
                None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), K.ERR_INVALID_ARG),
    (dict(batch=K.PAGED_MAX_BATCH + 1), K.ERR_INVALID_ARG),
    (dict(max_blocks=0), K.ERR_INVALID_ARG),
    (dict(max_blocks=2 ** 27), K.ERR_INVALID_ARG),               # 2^31 rows
    (dict(max_blocks=2 ** 26, batch=128), K.ERR_UNSUPPORTED),    # 2^32 steps
    (dict(q_stride=-8), K.ERR_INVALID_ARG),
    (dict(q_stride=1028), K.ERR_INVALID_ARG),
    (dict(scale=-1.0), K.ERR_INVALID_ARG),
    (dict(scale=math.inf), K.ERR_INVALID_ARG),
    (dict(softcap=-1.0), K.ERR_INVALID_ARG),
    (dict(softcap=math.nan), K.ERR_INVALID_ARG),
    (dict(window=-1), K.ERR_INVALID_ARG),
])
def test_bad_attend_descriptor(kw, status):
    base = dict(batch=2, max_blocks=4)
    base.update(kw)
    p = K.make_paged_attend_desc(**base)
    n = ctypes.c_size_t(0)
    assert _raw("kvsel_paged_attend_workspace_size", _cache(), p, ctypes.byref(n)) == status
    assert _raw("kvsel_paged_attend", _cache(), p, 16, 16, 32, 16, 16, None, None, None, 16, None, 256, BIG,
                None) == status


def test_attend_heads_and_pointers():
    p = K.make_paged_attend_desc(batch=2, max_blocks=4)
    n = ctypes.c_size_t(0)
    for d in (16, 96, 256):
        assert _raw("kvsel_paged_attend_workspace_size", _cache(head_dim=d), p, ctypes.byref(n)) == K.ERR_UNSUPPORTED

    def call(c=None, q=16, k=16, v=32, table=16, lens=16, slopes=None, ks=None, vs=None, o=16, lse=None, ws=256, nb=BIG):
        return _raw("kvsel_paged_attend", c or _cache(), p, q, k, v, table, lens, slopes, ks, vs, o, lse, ws, nb, None)
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(table=None), dict(lens=None), dict(o=None), dict(q=8),
               dict(k=8), dict(v=24), dict(o=8), dict(lens=4), dict(table=2), dict(slopes=2), dict(lse=2),
               dict(ks=16, vs=16), dict(ks=16), dict(c=_cache(cache_dtype=K.DTYPE_E4M3)),
               dict(c=_cache(cache_dtype=K.DTYPE_E4M3), ks=16)):
        assert call(**kw) == K.ERR_INVALID_ARG, kw
    assert call(ws=None) == K.ERR_WORKSPACE
    assert call(ws=128) == K.ERR_WORKSPACE


def test_append_arguments():
    def call(c=None, n=4, q=16, k=16, v=16, pos=16, slots=16, qw=None, kw=None, freq=16, qo=16, kc=16, vc=32, ks=None,
             vs=None, ws=None, strides=(1024, 128, 256, 128, 256, 128), **rope):
        r = K.make_rope_desc(**{**dict(rot_dim=128), **rope})
        (r.q_stride, r.q_head_stride, r.k_stride, r.k_head_stride, r.v_stride, r.v_head_stride) = strides
        return _raw("kvsel_rope_append", c or _cache(), r, n, q, k, v, pos, slots, qw, kw, freq, qo, kc, vc, ks, vs, ws,
                    None)
    e4 = _cache(cache_dtype=K.DTYPE_E4M3)
    for kw in (dict(n=-1), dict(n=2 ** 31), dict(rot_dim=144), dict(rot_dim=-16), dict(layout=2),
               dict(factor=math.nan), dict(norm_eps=-1.0), dict(weight_bias=math.inf), dict(q=None, qo=None, k=None,
               v=None, kc=None, vc=None), dict(qo=None), dict(q=None), dict(v=None), dict(kc=None), dict(vc=None),
               dict(slots=None), dict(pos=None), dict(freq=None), dict(q=8), dict(k=8), dict(vc=40), dict(qw=2),
               dict(pos=4), dict(slots=4), dict(freq=4), dict(kc=16, vc=16), dict(ks=16, vs=16), dict(c=e4),
               dict(c=e4, ks=16), dict(strides=(1028, 128, 256, 128, 256, 128)),
               dict(strides=(1024, 128, 256, 128, -256, 128)),
               dict(strides=(2048, 128, 256, 128, 256, 128))):           # in place over rows laid out otherwise
        assert call(**kw) == K.ERR_INVALID_ARG, kw
    assert call(rot_dim=24) == K.ERR_UNSUPPORTED
    assert call(ws=128) == K.ERR_WORKSPACE
    assert call(n=0) == K.OK                                             # nothing to do, nothing launched


def test_assign_arguments():
    n = ctypes.c_size_t(0)
    for b in (0, K.PAGED_MAX_BATCH + 1):
        assert K.raw_call("kvsel_page_assign_workspace_size", b, ctypes.byref(n)) == K.ERR_INVALID_ARG
    assert K.raw_call("kvsel_page_assign_workspace_size", 4, None) == K.ERR_INVALID_ARG
    assert K.kvsel_page_assign_workspace_size(4) % K.WS_ALIGN == 0

    def call(P=16, pages=100, batch=2, blocks=4, lens=16, new=16, off=None, free=16, n_free=10, head=16, table=16,
             lens_out=16, head_out=16, indptr=16, tokens=8, slots=16, pos=16, ids=16, ws=256, nb=BIG):
        return K.raw_call("kvsel_page_assign", P, pages, batch, blocks, lens, new, off, free, n_free, head, table,
                          lens_out, head_out, indptr, tokens, slots, pos, ids, ws, nb, None)
    for kw in (dict(P=0), dict(P=257), dict(pages=0), dict(pages=2 ** 31), dict(batch=0),
               dict(batch=K.PAGED_MAX_BATCH + 1), dict(blocks=0), dict(blocks=2 ** 27), dict(n_free=-1),
               dict(n_free=2 ** 31), dict(tokens=-1), dict(tokens=2 ** 31), dict(lens=None), dict(new=None),
               dict(head=None), dict(table=None), dict(lens_out=None), dict(head_out=None), dict(indptr=None),
               dict(free=None), dict(slots=None), dict(lens=4), dict(new=12), dict(off=4), dict(head=4), dict(slots=4),
               dict(pos=4), dict(free=2), dict(table=2), dict(ids=2)):
        assert call(**kw) == K.ERR_INVALID_ARG, kw
    for kw in (dict(ws=None), dict(ws=64), dict(nb=255)):
        assert call(**kw) == K.ERR_WORKSPACE, kw


def test_rope_freqs_against_the_definition():
    types = {"plain": K.ROPE_PLAIN, "linear": K.ROPE_LINEAR, "banded": K.ROPE_BANDED, "ramp": K.ROPE_RAMP}
    for kind, t in types.items():
        for rot in (2, 16, 64, 128):
            for base, factor, low, high, L0 in ((10000.0, 4.0, 1.0, 4.0, 8192), (500000.0, 8.0, 1.0, 32.0, 4096)):
                f, scale = K.kvsel_rope_freqs(rot, K.RopeScaling(t, base, factor, low, high, L0))
                want, ws = O.rope_freqs(rot, kind, base, factor, low, high, L0)
                np.testing.assert_allclose(f, want, rtol=1e-13)
                assert abs(scale - ws) <= 2.0 ** -24 * ws
    out, sc = (ctypes.c_double * 64)(), ctypes.c_float(0)
    good = (K.ROPE_RAMP, 10000.0, 4.0, 1.0, 4.0, 8192)
    for at, bad in ((0, 4), (0, -1), (1, 1.0), (1, math.inf), (2, 0.5), (2, math.nan), (3, 0.0), (4, 1.0), (5, 0)):
        s = K.RopeScaling(*[bad if i == at else x for i, x in enumerate(good)])
        assert K.raw_call("kvsel_rope_freqs", 128, ctypes.byref(s), out, ctypes.byref(sc)) == K.ERR_INVALID_ARG
    s = K.RopeScaling(*good)
    for rot in (0, 3, 258):
        assert K.raw_call("kvsel_rope_freqs", rot, ctypes.byref(s), out, ctypes.byref(sc)) == K.ERR_INVALID_ARG


def test_strided_heads_are_read_from_the_tensors():
    qkv = torch.zeros(5, 12, 64)
    r = K.make_rope_desc(rot_dim=64, q=qkv[:, :8], k=qkv[:, 8:10], v=qkv.transpose(1, 2)[:, :, :].transpose(1, 2)[:, 10:])
    assert (r.q_stride, r.q_head_stride, r.v_stride, r.v_head_stride) == (12 * 64, 64, 12 * 64, 64)
    with pytest.raises(ValueError):
        K.make_rope_desc(rot_dim=64, q=qkv.transpose(1, 2))


# ---- the definitions --------------------------------------------------------------------------------
def test_definition_of_attention_matches_sdpa():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((4, 64)), rng.standard_normal((37, 64)), rng.standard_normal((37, 64))
    tq, tk, tv = (torch.from_numpy(x)[None, None] for x in (q, k, v))
    o, lse, mass, _ = O.paged_attend(q, k, v, 0.125)
    want = torch.nn.functional.scaled_dot_product_attention(tq, tk, tv, scale=0.125)[0, 0]
    np.testing.assert_allclose(o, want.numpy(), rtol=1e-12)
    np.testing.assert_allclose(lse, torch.logsumexp(tq @ tk.transpose(-1, -2) * 0.125, -1)[0, 0].numpy(), rtol=1e-12)
    assert (mass >= np.abs(o) - 1e-12).all()
    slopes = np.array([0.5, 0.25, 0.125, 0.0625])
    o, *_ = O.paged_attend(q, k, v, 0.125, window=10, slopes=slopes)
    bias = torch.from_numpy(slopes)[:, None] * (torch.arange(37) - 36)
    bias = torch.where(torch.arange(37) >= 27, bias, -math.inf)[None, None]
    want = torch.nn.functional.scaled_dot_product_attention(tq, tk, tv, attn_mask=bias, scale=0.125)[0, 0]
    np.testing.assert_allclose(o, want.numpy(), rtol=1e-12)
    # a cap far above the scores changes nothing, a tiny one makes all rows equal
    np.testing.assert_allclose(O.paged_attend(q, k, v, 0.125, softcap=1e8)[0], O.paged_attend(q, k, v, 0.125)[0], rtol=1e-8)
    np.testing.assert_allclose(O.paged_attend(q, k, v, 0.125, softcap=1e-9)[0], np.tile(v.mean(0), (4, 1)), atol=1e-8)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_definition_of_rotation(layout):
    """Turned rows keep their length, and scores depend on the difference of positions alone."""
    rng = np.random.default_rng(4)
    f, _ = O.rope_freqs(32, "plain", 10000.0)
    x, y = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64))

    def at(v, p):
        return O.norm_rope(v, np.array([p]), f, 1.0, layout)[0][0, 0]
    np.testing.assert_allclose(np.linalg.norm(at(x, 12345)), np.linalg.norm(x), rtol=1e-12)
    np.testing.assert_allclose(at(x, 100) @ at(y, 93), at(x, 1007) @ at(y, 1000), rtol=1e-9)
    np.testing.assert_array_equal(at(x, 7)[32:], x[0, 0, 32:])
    pair = (0, 16) if layout == "half" else (0, 1)
    a, b = x[0, 0, pair[0]], x[0, 0, pair[1]]
    assert abs(at(x, 1)[pair[0]] - (a * math.cos(1) - b * math.sin(1))) < 1e-12
