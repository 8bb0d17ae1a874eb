"""Beam selection where scores are equal: the smaller beam, then the larger logit, then the smaller token; and many entries at -inf."""

import math

import pytest
import torch

from tests.test_gpu_beam_select import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from attention_kv_cache_gb300 import kvsel
    return kvsel


@pytest.mark.parametrize("spots", [[5, 9000, 17000], [17000, 5, 9000], [24575, 8192, 8191], [7, 6, 5]], ids=str)
def test_logits_apart_by_less_than_a_score(cuda, K, spots):
    """Logits of 1e-20 and its multiples, whose scores are one 64-bit number: the larger logit first, in whatever segment."""
    c = Case(K, cuda, 1, 2, 6, 3 * 8192, "f32")
    c.logits.fill_(-50.0)
    for i, t in enumerate(spots):
        c.logits[:, t] = (len(spots) - i) * 1e-20
    c.scores.copy_(torch.tensor([[-1.0, -3.0]]))
    c.run().check()
    assert c.tokens.tolist() == [spots * 2] and c.parents.tolist() == [[0, 0, 0, 1, 1, 1]]


@pytest.mark.parametrize("n_out", [1, 10, 64])
@pytest.mark.parametrize("score", [-1.0, 1e30])
def test_more_equal_heads_than_outputs(cuda, K, n_out, score):
    """100 segments to a row whose best logits differ, the largest in the last ones, all at one score."""
    c = Case(K, cuda, 1, 2, n_out, 100 * 8192, "f32")
    c.logits.fill_(-50.0)
    for i in range(100):
        c.logits[:, i * 8192 + 3 * i] = (i % 70 + 1) * 1e-20
    c.scores.fill_(score)
    c.run()
    torch.cuda.synchronize()
    order = sorted(range(100), key=lambda i: (-(i % 70), i))
    want = [i * 8192 + 3 * i for i in order]
    assert c.tokens[0].tolist() == want[:n_out] and c.parents[0].tolist() == [0] * n_out
    if score == 1e30:                                          # (every token of the vocabulary at one score)
        assert (c.out == torch.tensor(1e30, device=cuda)).all()
    else:
        assert (c.out - (-1.0 - math.log(100.0))).abs().max() < 2.0 ** -18


@pytest.mark.parametrize("beams,vocab", [(32, 20000), (64, 9000), (64, 300), (16, 40000)])
@pytest.mark.parametrize("live", [[0], [], [0, 5]], ids=["first", "none", "two"])
def test_a_wide_sets_first_step(cuda, K, beams, vocab, live):
    """Every beam but a few without a score, 64 outputs: what is left of them are the first beam's first tokens at -inf."""
    c = Case(K, cuda, 2, beams, 64, vocab, "bf16")
    c.logits[:beams, 40:] = float("-inf")                      # (in the first set the live beams have 40 tokens)
    dead = torch.ones(beams, dtype=torch.bool)
    dead[live] = False
    c.scores[:, dead] = float("-inf")
    c.run().check()
