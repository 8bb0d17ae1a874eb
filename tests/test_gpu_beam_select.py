"""Beam selection against the fp64 definition, sorted in Python.

Parents and tokens are equal.  A score is formed in 64 bits from a log-sum of exponentials that are within 2^-22 each and summed by
threads in fp32 (256 terms: 2^-16 of a sum's own at most, 2^-20 as they come), and rounded once: |score - ref| <= 2^-18 + 2^-24 |ref|.
The inputs of the tests leave more than that between scores of different beams, or none at all (the tests of ties).
"""

import numpy as np
import pytest
import torch

from oracle import paged_oracle as O
from tests import paged_common as C

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


class Case:
    def __init__(self, K, cuda, batch, beams, n_out, vocab, dtype="f32", pad=0, pad_token=0, offset=0):
        kinds = {"bf16": K.DTYPE_BF16, "f16": K.DTYPE_F16, "f32": K.DTYPE_F32}
        self.K, self.batch, self.beams, self.n_out, self.vocab, self.pad_token = K, batch, beams, n_out, vocab, pad_token
        g = torch.Generator().manual_seed(batch * 1000 + beams * 100 + vocab)
        rows = batch * beams
        store = torch.randn(rows * (vocab + pad) + offset, generator=g) * 2
        self.store = store.to(DT[dtype]).to(cuda)
        self.logits = self.store[offset:].view(rows, vocab + pad)[:, :vocab]
        self.scores = (-10 - 4 * torch.rand(batch, beams, generator=g)).to(cuda)
        self.ended = None
        self.desc = K.make_beam_select_desc(batch=batch, beams=beams, n_out=n_out, vocab=vocab, dtype=kinds[dtype],
                                            row_stride=vocab + pad, pad_token=pad_token)
        self.ws = C.workspace(K, K.kvsel_beam_select_workspace_size(self.desc), cuda)
        self.out = torch.full((batch, n_out), 7.0, device=cuda)
        self.parents, self.tokens = (torch.full((batch, n_out), -5, dtype=torch.int32, device=cuda) for _ in range(2))
        self.lse = torch.full((batch, beams), 7.0, device=cuda)

    def run(self, stream=None):
        self.K.kvsel_beam_select(self.desc, self.logits, self.scores, self.ended, self.out, self.parents, self.tokens, self.lse,
                                 self.ws, stream=stream)
        return self

    def check(self):
        torch.cuda.synchronize()
        x = self.logits.double().cpu().numpy().reshape(self.batch, self.beams, self.vocab)
        for b in range(self.batch):
            e = None if self.ended is None else self.ended[b].cpu().numpy()
            s, p, t, lse = O.beam_select(x[b], self.scores[b].double().cpu().numpy(), self.n_out, e, self.pad_token)
            assert np.array_equal(self.parents[b].cpu().numpy(), p), (b, self.parents[b], p)
            assert np.array_equal(self.tokens[b].cpu().numpy(), t), (b, self.tokens[b], t)
            for got, ref in ((self.out[b], s), (self.lse[b], lse)):
                got = got.double().cpu().numpy()
                fin = np.isfinite(ref)
                assert np.array_equal(got[~fin], ref[~fin])
                assert (np.abs(got[fin] - ref[fin]) <= 2.0 ** -18 + 2.0 ** -24 * np.abs(ref[fin])).all()
        return self


@pytest.fixture(scope="module")
def K():
    from attention_kv_cache_gb300 import kvsel
    return kvsel


@pytest.mark.parametrize("batch,beams,n_out,vocab", [
    (1, 1, 1, 1), (1, 1, 5, 5), (3, 2, 4, 7), (2, 4, 8, 8191), (2, 4, 8, 8192), (1, 4, 8, 8193), (1, 3, 6, 50003), (2, 64, 64, 300),
    (1, 64, 64, 64), (1, 1, 64, 20001), (40, 5, 10, 1000), (1, 2, 33, 9000),
])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_shapes(cuda, K, batch, beams, n_out, vocab, dtype):
    Case(K, cuda, batch, beams, n_out, vocab, dtype).run().check()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad,offset", [(1, 0), (3, 1), (5, 2), (0, 7), (8, 8), (64, 4)])
def test_rows_anywhere(cuda, K, dtype, pad, offset):
    """Row strides and first elements of every alignment; equal rows give equal bits wherever they lie."""
    c = Case(K, cuda, 2, 4, 8, 20000, dtype, pad=pad, offset=offset)
    c.logits[1:] = c.logits[0]
    c.scores[:] = c.scores[0, 0]
    c.run().check()
    assert (c.lse == c.lse[0, 0]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ties_go_to_the_smaller_beam_and_token(cuda, K, dtype):
    for values in (torch.zeros(1), torch.arange(5.0), torch.tensor([3.0, -1.0])):
        c = Case(K, cuda, 2, 3, 20, 9001, dtype)
        c.logits.copy_(values.to(c.logits)[torch.arange(9001, device=cuda) % len(values)].expand_as(c.logits))
        c.scores.fill_(-2.0)
        c.run().check()


def test_rising_and_falling_logits(cuda, K):
    """Every slice passes the bound of the ones before it, and none does."""
    for sign in (1, -1):
        c = Case(K, cuda, 1, 1, 64, 65536, "f32")
        c.logits.copy_(sign * torch.arange(65536, device=cuda).float() / 4096)
        c.run().check()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_tokens_that_are_not_allowed(cuda, K, dtype):
    """Most of a vocabulary at -inf, rows of nothing else, NaN and +inf among the logits."""
    c = Case(K, cuda, 2, 4, 12, 30000, dtype)
    keep = torch.zeros(30000, dtype=torch.bool)
    keep[[5, 8191, 8192, 17000, 29999]] = True
    c.logits[:4, ~keep] = float("-inf")
    c.logits[5] = float("-inf")
    c.logits[6, 77] = float("nan")
    c.logits[6, 29000:29040] = float("nan")
    c.logits[7, 123] = float("inf")
    c.run().check()


def test_ended_and_empty_beams(cuda, K):
    c = Case(K, cuda, 4, 5, 12, 4000, "bf16", pad_token=7)
    c.ended = torch.zeros(4, 5, dtype=torch.uint8, device=cuda)
    c.ended[0, 1] = 1
    c.ended[1] = 1
    c.scores[2, 1:] = float("-inf")
    c.scores[3] = float("-inf")
    c.ended[3, 2] = 1
    c.scores[0, 3] = float("nan")
    c.scores[0, 4] = float("inf")
    c.run().check()


def test_one_token_of_a_small_vocabulary(cuda, K):
    c = Case(K, cuda, 3, 4, 8, 2, "f16", pad_token=1)
    c.ended = torch.tensor([[0, 1, 0, 1]] * 3, dtype=torch.uint8, device=cuda)
    c.run().check()


def test_rows_of_one_tensor(cuda, K):
    """All beams over the same logits (stride 0 is the vocabulary's: an expanded tensor is copied by its user)."""
    c = Case(K, cuda, 1, 4, 8, 5000, "bf16")
    c.logits.copy_(c.logits[0].clone().expand_as(c.logits))
    c.run().check()


def test_streams_and_capture(cuda, K):
    c = Case(K, cuda, 3, 4, 8, 12345, "bf16", pad=2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.run(stream=side)
    side.synchronize()
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for seed in (1, 2):
        c.logits.copy_(torch.randn(c.logits.shape, generator=torch.Generator().manual_seed(seed)) * 3)
        g.replay()
        c.check()
