"""The calls for chunks, prefixes and beams stay inside their buffers: every output and the workspace lie in guard regions of a known
pattern, at sizes that leave every tile, page and box partly filled."""

import numpy as np
import pytest
import torch

from tests.test_gpu_beam_reorder import Case as Reorder
from tests.test_gpu_beam_select import Case as Select
from tests.test_gpu_chunk_attend import Case as Chunk
from tests.test_gpu_paged_guards import Guarded
from tests.test_gpu_prefix_attend import Case as Prefix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from attention_kv_cache_gb300 import kvsel
    return kvsel


@pytest.mark.parametrize("kw", [
    dict(held=[0, 5, 300], new=[1, 130, 33]), dict(held=[0], new=[1], pad=0), dict(held=[77, 9], new=[100, 200], d=64, G=7, P=9),
    dict(held=[500] * 30, new=[3] * 30, cache="e4m3", P=24, order="row"), dict(held=[2000, 1], new=[40, 1], cache="e4m3", P=5, dtype="f16"),
], ids=range(5))
def test_chunk(cuda, K, kw):
    c, g = Chunk(K, cuda, **kw), Guarded(cuda)
    c.o, c.lse, c.ws = g.put(c.o), g.put(c.lse, 4), g.put(c.ws)
    c.run().check()
    g.check()


@pytest.mark.parametrize("kw", [
    dict(groups=[(100, [1, 2, 3])]), dict(groups=[(16, [0])], d=64), dict(groups=[(600, [5] * 50), (0, [9]), (33, [])], cache="e4m3", P=9),
    dict(groups=[(200, [1] * 9)] * 9, G=3, h_kv=1, dtype="f16", order="row"),
], ids=range(4))
def test_prefix(cuda, K, kw):
    c, g = Prefix(K, cuda, **kw), Guarded(cuda)
    c.o, c.lse, c.ws = g.put(c.o), g.put(c.lse, 4), g.put(c.ws)
    c.run().check()
    g.check()


@pytest.mark.parametrize("args", [(1, 1, 1, 1), (3, 5, 10, 20001, "bf16", 1), (2, 64, 64, 100, "f16"), (5, 3, 6, 8193, "f32", 3)], ids=range(4))
def test_select(cuda, K, args):
    c, g = Select(K, cuda, *args), Guarded(cuda)
    c.out, c.parents, c.tokens, c.lse, c.ws = (g.put(x, a) for x, a in ((c.out, 4), (c.parents, 4), (c.tokens, 4), (c.lse, 4), (c.ws, 256)))
    c.run().check()
    g.check()


@pytest.mark.parametrize("kw", [dict(lens=[1], beams=1), dict(lens=[100, 33, 0], beams=5), dict(lens=[2049, 70], beams=3, P=7, cache="e4m3"),
                                dict(lens=[300] * 9, beams=8, order="row", cache="f16")], ids=range(4))
def test_reorder(cuda, K, kw):
    c, g = Reorder(K, cuda, in_place=False, **kw), Guarded(cuda)
    c.to, c.lo, c.ho, c.f, c.ws = (g.put(x, a) for x, a in ((c.to, 4), (c.lo, 8), (c.ho, 8), (c.f, 4), (c.ws, 256)))
    c.pools = [g.put(x) for x in c.pools]
    rng = np.random.default_rng(1)
    c.run([rng.integers(0, c.beams, c.beams).tolist() for _ in kw["lens"]]).check()
    g.check()
