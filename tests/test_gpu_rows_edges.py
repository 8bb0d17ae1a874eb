"""Attention of many rows at the ends of its range."""

import pytest

from tests.test_gpu_chunk_attend import Case as Chunk
from tests.test_gpu_prefix_attend import Case as Prefix

pytestmark = pytest.mark.gpu


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
