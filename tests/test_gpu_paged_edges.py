"""Attention at the ends of its descriptors' ranges."""

import pytest
import torch

from tests.test_gpu_paged_attend import Case

pytestmark = pytest.mark.gpu


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
