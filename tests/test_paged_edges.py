"""Ends of the paged calls' ranges that are decided on the host (no GPU)."""

import ctypes
import math

import pytest
import torch

from attention_kv_cache_gb300 import kvsel as K


@pytest.mark.parametrize("kv", [True, False])
@pytest.mark.parametrize("queries", [True, False])
@pytest.mark.parametrize("cache_dtype", [K.DTYPE_BF16, K.DTYPE_E4M3])
def test_a_step_of_no_tokens_has_nothing_to_append(queries, kv, cache_dtype):
    """Tensors of no tokens have no address, which is not an argument left out."""
    c = K.make_cache_desc(h_q=8, h_kv=2, head_dim=64, page_size=16, n_pages=4, cache_dtype=cache_dtype)
    x = torch.empty(0, 12, 64, dtype=torch.bfloat16)
    q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
    empty = torch.empty(0, dtype=torch.int64)
    assert x.data_ptr() == 0
    r = K.make_rope_desc(rot_dim=64, q=q, k=k, v=v)
    K.kvsel_rope_append(c, r, q if queries else None, k if kv or not queries else None, v if kv or not queries else None,
                        empty, empty, None, None, 16, torch.empty(0, 8, 64) if queries else None, 16 if kv else None,
                        32 if kv else None, 16 if kv else None, 16 if kv else None, stream=0)
    r.rot_dim = 65                                       # the descriptors are checked all the same
    with pytest.raises(K.KvselError):
        K.kvsel_rope_append(c, r, q, k, v, empty, empty, None, None, 16, q, 16, 32, stream=0)


def _attend_size(**kw):
    c = K.make_cache_desc(h_q=8, h_kv=2, head_dim=128, page_size=16, n_pages=4)
    p = K.make_paged_attend_desc(batch=2, max_blocks=4, **kw)
    n = ctypes.c_size_t(0)
    return K.raw_call("kvsel_paged_attend_workspace_size", ctypes.byref(c), ctypes.byref(p), ctypes.byref(n))


def test_caps_that_fp32_cannot_divide_by_are_refused():
    """Below 2^-126 the reciprocal is infinite, and 0 of it no number; above 2^127 the cap in base 2 is infinite."""
    for cap in (2.0 ** -127, 1e-45, 1.5 * 2.0 ** 127, math.inf, -math.inf, math.nan, -1.0):
        assert _attend_size(softcap=cap) == K.ERR_INVALID_ARG, cap
    for cap in (0.0, 2.0 ** -126, 2.0 ** 127):
        assert _attend_size(softcap=cap) in (K.OK, K.ERR_CUDA), cap        # (without a GPU its SMs cannot be asked for)
