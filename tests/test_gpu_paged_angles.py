"""Rotary angles at far positions, against angles formed in whole numbers.

The exact angle of a position and a frequency (a double, hence a fraction) is position * frequency modulo 2 pi, with pi to
400 bits.  Tolerances are those of tests/test_gpu_paged_append.py: 2^-18 (|a| + |b|) of a turned pair, for the cosine, the sine
and the arithmetic, and half a step of the output.
"""

from fractions import Fraction

import numpy as np
import pytest
import torch

from tests import paged_common as C
from tests.test_gpu_paged_append import near

pytestmark = pytest.mark.gpu
ONE = 1 << 400


def _arctan_of_inverse(x):
    """arctan(1 / x) as a multiple of 1 / ONE, by its series."""
    term, n, sign = ONE // x, 1, 1
    total = 0
    while term:
        total += sign * (term // n)
        term, n, sign = term // (x * x), n + 2, -sign
    return total


TWO_PI = Fraction(2 * 4 * (4 * _arctan_of_inverse(5) - _arctan_of_inverse(239)), ONE)


def angles(pos, freq):
    """position * frequency modulo 2 pi, in (-pi, pi], as doubles."""
    turns = [Fraction(float(f)) / TWO_PI for f in freq]
    out = np.empty((len(pos), len(freq)))
    for i, p in enumerate(pos):
        for j, t in enumerate(turns):
            x = (int(p) * t) % 1
            out[i, j] = float((x - 1 if x > Fraction(1, 2) else x) * TWO_PI)
    return out


def rotate(cuda, q, pos, freq, layout="half"):
    """Queries [n, h, d] turned at `pos`, as doubles."""
    from attention_kv_cache_gb300 import kvsel as K
    n, h, d = q.shape
    kind = {v: k for k, v in C.DT.items()}[q.dtype]
    desc = K.make_cache_desc(h_q=h, h_kv=h, head_dim=d, page_size=16, n_pages=1, dtype=C.kinds(K)[kind])
    out, qd = torch.empty_like(q, device=cuda), q.to(cuda)
    K.kvsel_rope_append(desc, K.make_rope_desc(rot_dim=2 * len(freq), layout=K.ROPE_HALF if layout == "half" else K.ROPE_INTERLEAVED,
                                               q=qd), qd, None, None, torch.as_tensor(pos, device=cuda), None, None, None,
                        torch.as_tensor(freq, device=cuda), out, None, None)
    torch.cuda.synchronize()
    return C.f64(out)


POSITIONS = np.array([0, 1, 2 ** 20, 2 ** 23 + 1, 2 ** 27 - 5, 2 ** 29 + 12345, 2 ** 30 + 987654321 % 2 ** 30, 2 ** 31 - 1] +
                     [x * 33554393 % 2 ** 31 for x in range(1, 41)])


def test_pi():
    assert float(TWO_PI / 2) == np.pi and abs(float(Fraction(np.sin(1e-9)) - Fraction(1, 10 ** 9))) < 1e-25


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("top", [1.0, 50.0, 3e3, 1e6, 1e9])
def test_any_frequency_at_any_position(cuda, top, layout):
    """The turn of a pair is kept to 2^-32 of a turn at 2^31 positions, however often the pair turns per position."""
    g = torch.Generator().manual_seed(2)
    d, n = 64, len(POSITIONS)
    freq = top ** (1 - np.arange(d // 2) / (d // 2)) * (1 + 0.1 * torch.rand(d // 2, generator=g).double().numpy())
    q = torch.randn(n, 2, d, generator=g).half()
    angle = angles(POSITIONS, freq)[:, None]
    x = C.f64(q)
    a, b = (x[..., :d // 2], x[..., d // 2:]) if layout == "half" else (x[..., 0::2], x[..., 1::2])
    y = np.empty_like(x), np.empty_like(x)
    first, second = (slice(0, d // 2), slice(d // 2, d)) if layout == "half" else (slice(0, d, 2), slice(1, d, 2))
    y[0][..., first], y[0][..., second] = a * np.cos(angle) - b * np.sin(angle), b * np.cos(angle) + a * np.sin(angle)
    y[1][..., first] = y[1][..., second] = np.abs(a) + np.abs(b)
    near(rotate(cuda, q, POSITIONS, freq, layout), *y, "f16", "turned")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_cosines_and_sines_to_2_22(cuda, layout):
    """Pairs of whole numbers with a cos ~ b sin: what is left of the turned pair shows the cosine's and the sine's errors.

    With each off by at most 2^-22, a cos rounded (2^-24 |a|) and everything else exact or a rounding of the small result, the
    result is off by 2^-22 (|a| + |b|) + 2^-24 |a| and half a step of its own."""
    d = 256
    freq = 500000.0 ** (-np.arange(d // 2) / (d // 2))
    angle = angles(POSITIONS, freq)
    cos, sin = np.cos(angle), np.sin(angle)
    many = np.arange(1024, 2048)[:, None, None]
    steep = np.abs(sin) > np.abs(cos)                     # the larger of the two numbers is `many`, the other follows
    other = np.rint(many * np.where(steep, cos / np.where(steep, sin, 1.0), sin / np.where(steep, 1.0, cos)))
    a, b = np.where(steep, many, other), np.where(steep, other, many)
    best = np.abs(a * cos - b * sin).argmin(0)[None]
    a, b = (np.take_along_axis(x, best, 0)[0] for x in (a, b))
    q = torch.empty(len(POSITIONS), 1, d, dtype=torch.half)
    first, second = (slice(0, d // 2), slice(d // 2, d)) if layout == "half" else (slice(0, d, 2), slice(1, d, 2))
    q[:, 0, first], q[:, 0, second] = torch.from_numpy(a).half(), torch.from_numpy(b).half()
    assert np.array_equal(C.f64(q[:, 0, first]), a) and np.array_equal(C.f64(q[:, 0, second]), b)
    got = rotate(cuda, q, POSITIONS, freq, layout)[:, 0]
    for part, want, mul in ((first, a * cos - b * sin, a), (second, b * cos + a * sin, b)):
        tol = 2.0 ** -22 * (np.abs(a) + np.abs(b)) + 2.0 ** -24 * np.abs(mul)
        tol += 2.0 ** -11 * (np.abs(want) + tol) + 2.0 ** -25
        bad = ~(np.abs(got[:, part] - want) <= tol)
        assert not bad.any(), (bad.sum(), (np.abs(got[:, part] - want) / tol).max())
