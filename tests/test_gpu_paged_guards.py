"""The paged calls stay inside their buffers: every output and the workspace lie in guard regions of a known pattern,
at sizes that leave every tile, page and box partly filled."""

import pytest
import torch

from tests import paged_common as C
from tests.test_gpu_paged_append import Case as Append
from tests.test_gpu_paged_assign import Case as Assign
from tests.test_gpu_paged_attend import Case as Attend

pytestmark = pytest.mark.gpu
GUARD = 4096


class Guarded:
    """Copies of tensors inside one buffer, with GUARD bytes of a pattern around each."""

    def __init__(self, cuda):
        self.cuda, self.parts = cuda, []

    def put(self, t, align=256):
        n = t.numel() * t.element_size()
        buf = torch.full((n + 2 * GUARD + align,), 0xA5, dtype=torch.uint8, device=self.cuda)
        off = GUARD + (-(buf.data_ptr() + GUARD)) % align
        view = buf[off:off + n].view(t.dtype).view(t.shape)
        view.copy_(t) if t.element_size() > 1 else view.view(torch.uint8).copy_(t.view(torch.uint8))
        self.parts.append((buf, off, n))
        return view

    def check(self):
        for i, (buf, off, n) in enumerate(self.parts):
            assert (buf[:off] == 0xA5).all() and (buf[off + n:] == 0xA5).all(), i


@pytest.mark.parametrize("kw", [
    dict(lens=[0, 1, 45, 333]), dict(lens=[7000, 13], G=8), dict(lens=[100] * 90 + [0] + [900], h_kv=8, G=4, d=64),
    dict(lens=[77, 1200], cache="e4m3", P=9), dict(lens=[77, 1200], G=20, h_kv=1, dtype="f16", order="row"),
], ids=range(5))
def test_attention(cuda, kw):
    from attention_kv_cache_gb300 import kvsel as K
    c, g = Attend(K, cuda, **kw), Guarded(cuda)
    c.o, c.lse, c.ws = g.put(c.o), g.put(c.lse), g.put(c.ws)
    c.pools = [g.put(p) for p in c.pools]
    c.run().check()
    g.check()


@pytest.mark.parametrize("kw", [
    dict(n=1), dict(n=37, pad=5, P=7), dict(n=501, cache="e4m3", h_q=5, h_kv=5, d=80), dict(n=64, dtype="f16", order="row",
    layout="interleaved", rot=32), dict(n=33, d=16, h_q=1, h_kv=1),
], ids=range(5))
def test_append(cuda, kw):
    from attention_kv_cache_gb300 import kvsel as K
    c, g = Append(K, cuda, **kw), Guarded(cuda)
    c.q_out, c.ws = g.put(c.q_out), g.put(c.ws)
    c.pools = [g.put(p) for p in c.pools]
    c.run().check()
    g.check()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("new", [[1, 0, 40], [5000, 1, 7]])
def test_assignment(cuda, new, in_place):
    from attention_kv_cache_gb300 import kvsel as K
    c, g = Assign(K, cuda, [16, 0, 31], new, pad=3), Guarded(cuda)
    for k in ("lens_out", "head_out", "indptr", "slots", "pos", "ids", "tables", "lens", "head"):
        c.d[k] = g.put(c.d[k])
    c.ws = g.put(c.ws)
    c.run(in_place).check()
    g.check()


def test_with_tracing_on(cuda):
    """Events around every launch change nothing, and name the kernels."""
    from attention_kv_cache_gb300 import kvsel as K
    a, p, s = Attend(K, cuda, [3000, 5]), Append(K, cuda, 50), Assign(K, cuda, [5, 6], [1, 5000])
    torch.cuda.synchronize()
    K.kvsel_trace_enable(True)
    try:
        a.run()
        p.run()
        s.run(in_place=True)
        names = K.kvsel_trace_read()
    finally:
        K.kvsel_trace_enable(False)
    assert {"paged_attend", "paged_join", "rope_append", "page_assign", "page_assign_fill"} <= set(names)
    assert all(n == 1 and ms >= 0 for n, ms in (names[k] for k in ("paged_attend", "rope_append")))
    a.check()
    p.check()
    s.check()


def test_calls_read_what_the_last_kernel_wrote(cuda):
    """Launches may overlap the drain of the kernel before them: inputs written just before each call are seen."""
    from attention_kv_cache_gb300 import kvsel as K
    c = Attend(K, cuda, [500, 2000], seed=3)
    want_q, lens = c.q.clone(), c.l.clone()
    for _ in range(30):
        c.qs.zero_()
        c.l.zero_()
        c.q.copy_(want_q)
        c.l.copy_(lens)
        c.run()
        out = c.o.clone()
        c.o.zero_()
    c.o.copy_(out)
    c.check()
    a = Append(K, cuda, 300)
    q = a.q.clone()
    for _ in range(30):
        a.q.zero_()
        a.q_out.zero_()
        a.q.copy_(q)
        a.run()
    a.check()
