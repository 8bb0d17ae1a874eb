"""Beam selection over vocabularies as long as its checks allow."""

import math

import pytest
import torch

from tests import paged_common as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from attention_kv_cache_gb300 import kvsel
    return kvsel


def test_a_row_of_more_than_2_to_the_24_tokens(cuda, K):
    """2048 rows over one buffer (a row stride of 8 elements), each of 2049 slices: a sum of 2^24 equal terms and more."""
    batch, vocab, stride = 2048, 2049 * 8192, 8
    store = torch.zeros(vocab + batch * stride, dtype=torch.bfloat16, device=cuda)
    desc = K.make_beam_select_desc(batch=batch, beams=1, n_out=2, vocab=vocab, dtype=K.DTYPE_BF16, row_stride=stride)
    ws = C.workspace(K, K.kvsel_beam_select_workspace_size(desc), cuda)
    out, lse = torch.empty(batch, 2, device=cuda), torch.empty(batch, 1, device=cuda)
    parents, tokens = (torch.empty(batch, 2, dtype=torch.int32, device=cuda) for _ in range(2))
    K.kvsel_beam_select(desc, store, torch.zeros(batch, 1, device=cuda), None, out, parents, tokens, lse, ws)
    torch.cuda.synchronize()
    # (threads add 32 ones a slice in fp32, exactly; a log of 16.6 is rounded once, by 2^-20, and was off by 2^-50)
    for got, want in ((lse, math.log(vocab)), (out, -math.log(vocab))):
        assert (got.double() - want).abs().max() <= 2.0 ** -20 * (1 + 2.0 ** -20)
    assert (tokens == torch.tensor([0, 1], device=cuda)).all()
