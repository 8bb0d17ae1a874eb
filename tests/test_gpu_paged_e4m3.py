"""Rows written into an e4m3 pool: values that lie between two e4m3 numbers.

x / scale of a value t scale, with t the exact middle of two e4m3 neighbours, is t itself in fp32 (the quotient is
representable, so a correctly rounded division returns it) and has to be held as the even neighbour.  The values are
products of a 5-bit t and a 6-bit scale: exact in fp16.
"""

import pytest
import torch

from tests import paged_common as C

pytestmark = pytest.mark.gpu


def middles():
    """Middles of neighbouring e4m3 numbers in fourteen binades (112 of them), either sign in turn."""
    t = torch.cat([torch.arange(17, 32, 2).float() * 2.0 ** e for e in range(-10, 4)])
    t[1::2] *= -1
    return t


def test_the_reference_rounds_to_even():
    t = torch.tensor([1.0625, 1.1875, 17.0, 19.0, -1.0625, -19.0])
    assert t.to(torch.float8_e4m3fn).float().tolist() == [1.0, 1.25, 16.0, 20.0, -1.0, -20.0]


@pytest.mark.parametrize("order", ["head", "row"])
@pytest.mark.parametrize("n", [1, 40])
def test_middles_go_to_the_even_neighbour(cuda, n, order):
    from attention_kv_cache_gb300 import kvsel as K
    t = middles()
    scale = torch.arange(3, 64, 2).float() / 64                        # one per KV head
    h_kv, d, P = len(scale), len(t), 16
    x = (t * scale[:, None]).half()
    assert torch.equal(x.float() / scale[:, None], t.expand(h_kv, -1)) # exact in fp16, and so are the quotients
    x = x.expand(n, -1, -1).contiguous().to(cuda)
    n_pages = -(-n // P)
    pools = [C.empty_pool(n_pages, P, h_kv, d, order, torch.float8_e4m3fn, cuda) for _ in range(2)]
    desc = K.make_cache_desc(h_q=h_kv, h_kv=h_kv, head_dim=d, page_size=P, n_pages=n_pages, dtype=K.DTYPE_F16,
                             cache_dtype=K.DTYPE_E4M3, order=K.ORDER_HEAD if order == "head" else K.ORDER_ROW)
    s = scale.to(cuda)
    K.kvsel_rope_append(desc, K.make_rope_desc(rot_dim=0, k=x, v=x), None, x, x, None, torch.arange(n, device=cuda),
                        None, None, None, None, pools[0], pools[1], s, s)
    torch.cuda.synchronize()
    want = t.to(torch.float8_e4m3fn).float()
    for pool in pools:
        got = C.pool_view(pool.view(torch.uint8), order).reshape(-1, h_kv, d)[:n].cpu().view(torch.float8_e4m3fn).float()
        bad = got != want
        assert not bad.any(), (bad.sum(), got[bad][:4], want.expand_as(got)[bad][:4])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_values_are_those_of_a_rounded_quotient(cuda, dtype):
    """Any values and scales: the e4m3 number nearest to the fp32 quotient, bit for bit (rows that neither turn nor norm)."""
    from attention_kv_cache_gb300 import kvsel as K
    g = torch.Generator().manual_seed(6)
    n, h_kv, d, P = 300, 8, 128, 16
    scale = torch.cat([0.01 + 0.01 * torch.rand(5, generator=g), torch.tensor([2.0 ** -30, 1e-3, 77.7])])
    mul = torch.tensor([1.0, 1.0, 4.0, 0.01, 1.0, 2.0 ** -24, 1.0, 300.0])
    x = (torch.randn(n, 2 * h_kv, d, generator=g) * mul.repeat(2)[:, None]).to(C.DT[dtype])
    x[0, :, :3] = torch.tensor([float("inf"), -float("inf"), 0.0])
    n_pages = -(-n // P)
    pools = [C.empty_pool(n_pages, P, h_kv, d, "row", torch.float8_e4m3fn, cuda) for _ in range(2)]
    kk = C.kinds(K)
    desc = K.make_cache_desc(h_q=h_kv, h_kv=h_kv, head_dim=d, page_size=P, n_pages=n_pages, dtype=kk[dtype],
                             cache_dtype=K.DTYPE_E4M3, order=K.ORDER_ROW)
    xd, s = x.to(cuda), scale.to(cuda)
    k, v = xd[:, :h_kv], xd[:, h_kv:]
    K.kvsel_rope_append(desc, K.make_rope_desc(rot_dim=0, k=k, v=v), None, k, v, None, torch.arange(n, device=cuda),
                        None, None, None, None, pools[0], pools[1], s, s)
    torch.cuda.synchronize()
    want = (x.float() / scale.repeat(2)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    for i, pool in enumerate(pools):
        got = pool.view(torch.uint8).reshape(-1, h_kv, d)[:n].cpu()
        assert torch.equal(got, want[:, i * h_kv:(i + 1) * h_kv])


@pytest.mark.parametrize("scale", [0.01, 1.0, 77.0, 2.0 ** -59, 2.0 ** -62, 1e-30, 2.0 ** 59, 2.0 ** 62, 1e30, -0.01])
@pytest.mark.parametrize("turned", [False, True])
def test_quotients_of_any_size(cuda, scale, turned):
    """Finite values whose quotient passes fp32 end at +-448 like infinities, tiny ones at zero, and NaN stays."""
    from attention_kv_cache_gb300 import kvsel as K
    g = torch.Generator().manual_seed(7)
    n, h_kv, d, P = 20, 2, 64, 16
    big = torch.tensor([3e38, 1e38, 1e30, 449.0, 448.0, 17.0, 1.0, 1e-3, 1e-30, 1e-38, 0.0, float("inf"), float("nan")])
    x = torch.cat([big, -big, torch.randn(d - 26, generator=g)]).bfloat16().expand(n, h_kv, d).contiguous().to(cuda)
    pools = [C.empty_pool(2, P, h_kv, d, "row", torch.float8_e4m3fn, cuda) for _ in range(2)]
    desc = K.make_cache_desc(h_q=h_kv, h_kv=h_kv, head_dim=d, page_size=P, n_pages=2, cache_dtype=K.DTYPE_E4M3,
                             order=K.ORDER_ROW)
    s = torch.full((h_kv,), scale, device=cuda)
    zero = torch.zeros(n, dtype=torch.int64, device=cuda)              # position 0: cosines 1 and sines 0
    freq = torch.ones(d // 2, dtype=torch.float64, device=cuda)
    K.kvsel_rope_append(desc, K.make_rope_desc(rot_dim=0 if not turned else d, k=x, v=x), None, x, x, zero if turned else None,
                        torch.arange(n, device=cuda), None, None, freq if turned else None, None, pools[0], pools[1], s, s)
    torch.cuda.synchronize()
    want = (x.float().cpu() / s.cpu()[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).float()
    for i, pool in enumerate(pools):
        if turned and i == 0:
            continue                                                   # (0 times an infinity is NaN in a turned pair)
        got = pool.view(torch.uint8).reshape(-1, h_kv, d)[:n].cpu().view(torch.float8_e4m3fn).float()
        same = (got == want) | (got.isnan() & want.isnan())
        assert same.all(), (x.cpu()[~same][:5], got[~same][:5], want[~same][:5])
