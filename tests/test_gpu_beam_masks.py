"""Beam selection over logits that are masked with large finite values, as samplers forbid tokens, and over large logits.

Tolerances are those of the selection's own tests (parents and tokens equal, scores and log-sums within 2^-18 + 2^-24 of themselves):
a token that is masked adds nothing to a sum that holds another, and rows of masks alone are sums of ones.  The allowed logits and
the beams' scores leave more than that between scores that are not equal.
"""

import numpy as np
import pytest
import torch

from oracle import paged_oracle as O
from tests.test_gpu_beam_select import DT, Case

pytestmark = pytest.mark.gpu
MASKS = [(d, m) for d in ("f32", "bf16") for m in (-1e4, -1e9, -1e10, -1e20, -1e30, -1e38, "lowest")] + [("f16", "lowest"), ("f16", -1e4)]


@pytest.fixture(scope="module")
def K():
    from attention_kv_cache_gb300 import kvsel
    return kvsel


def mask_value(dtype, m):
    return torch.finfo(DT[dtype]).min if m == "lowest" else m


def check_sets(c, sets):
    """Case.check of some sets."""
    torch.cuda.synchronize()
    x = c.logits.view(c.batch, c.beams, -1)[sets].double().cpu().numpy()
    for i, b in enumerate(sets):
        s, p, t, lse = O.beam_select(x[i], c.scores[b].double().cpu().numpy(), c.n_out, None, c.pad_token)
        for got, ref in ((c.out[b], s), (c.lse[b], lse)):
            assert (np.abs(got.double().cpu().numpy() - ref) <= 2.0 ** -18 + 2.0 ** -24 * np.abs(ref)).all(), (b, got, ref)
        assert np.array_equal(c.parents[b].cpu().numpy(), p) and np.array_equal(c.tokens[b].cpu().numpy(), t), b


@pytest.mark.parametrize("dtype,mask", MASKS)
@pytest.mark.parametrize("allowed", [[5], [5, 900], [0, 8191, 8192, 29999], list(range(29990, 30000)), []], ids=["one", "two", "ends", "last", "none"])
def test_few_tokens_are_allowed(cuda, K, dtype, mask, allowed):
    """An odd and an even number of threads whose tokens are all masked, slices of masks alone before and behind, rows of nothing else."""
    c = Case(K, cuda, 2, 3, 4, 30000, dtype)
    keep = torch.zeros(30000, dtype=torch.bool)
    keep[allowed] = True
    c.logits[:, ~keep] = mask_value(dtype, mask)
    c.run().check()


@pytest.mark.parametrize("dtype,mask", MASKS)
def test_masks_in_segments_of_several_slices(cuda, K, dtype, mask):
    """Rows enough that a CTA takes a whole row, slice after slice: masks first, between and last."""
    c = Case(K, cuda, 512, 4, 6, 20000, dtype)
    rows = c.logits.view(512, 4, -1)
    m = mask_value(dtype, mask)
    for b, (lo, hi) in enumerate([(0, 8192), (8192, 16384), (16384, 20000), (0, 19990), (10, 20000), (0, 20000), (0, 9000), (40, 8200)]):
        rows[b, :, lo:hi] = m
    c.run()
    check_sets(c, [0, 1, 2, 3, 4, 5, 6, 7, 8, 511])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("top", [1e7, 1e10, 1e30, 3e38])
def test_large_logits(cuda, K, dtype, top):
    """One logit far above the others, and rows of large logits alone."""
    c = Case(K, cuda, 2, 3, 3, 20000, dtype)
    c.logits[:3, 17] = top
    c.logits[3:, :] = top
    c.run().check()


def test_a_few_masked_rows_of_a_set(cuda, K):
    """Beams whose rows are masked throughout beside others that are not."""
    c = Case(K, cuda, 3, 4, 12, 9000, "f32")
    c.logits[1] = torch.finfo(torch.float32).min
    c.logits[6] = -1e30
    c.logits[8:11] = -1e10
    c.run().check()
