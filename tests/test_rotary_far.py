"""Angles at far positions and of large frequencies, against turns in whole numbers.

Tolerance. The angle keeps 2^-60 of a turn a position; its sine and cosine and what follows are as in test_rotary.
"""
import math
from fractions import Fraction

import pytest
import torch

from moe_decode_megakernel_02_gb300 import rotary
from test_latent import ints
from test_rotary import expected

gpu = pytest.mark.gpu
TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097")
FREQ = [1.0, 0.75, 0.731, 6.5, 10.0, 100.0, -100.5, 3.0e4, 1.0e6, -1e-9, 2.0 ** 40 + 1, 1e-30, 0.1, -0.3]


def angles(freq, at):
    """radians of the turns' fractions"""
    turns = [float((Fraction(f) * at / TWO_PI) % 1) for f in freq.tolist()]
    return torch.tensor(turns, dtype=torch.float64, device="cuda") * (2 * math.pi)


@gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("at", [3, -77, 123456789, (1 << 31) - 1, -(1 << 31)])
def test_angles_keep_their_turns(at, layout):
    g = torch.Generator(device="cuda").manual_seed(2)
    freq = torch.tensor(FREQ, dtype=torch.float64, device="cuda")
    x = torch.randn((1, 1, 5, 2 * len(FREQ)), generator=g, device="cuda")
    want, size = expected(x, torch.ones((1, 1), device="cuda"), angles(freq, at), layout, 0)
    got = rotary.rotate(x, ints(at), freq, layout=layout)
    slack = abs(at) * 2.0 ** -60 * 2 * math.pi
    err = (got.double() - want).abs()
    assert (err <= size * (2.0 ** -21 + slack) + want.abs() * 2.0 ** -21).all(), (err / size).amax((0, 1, 2))


@gpu
def test_rows_into_a_cache_keep_their_turns():
    """A cache has at most 2^30 positions, of which a table of few columns holds the last ones of few pages: the largest
    position here is 2^27."""
    cols, ps = 1 << 11, 1 << 16
    latent = torch.zeros((1, 1, 512), dtype=torch.float16, device="cuda")
    rope = torch.zeros((1, 1, 64), dtype=torch.float16, device="cuda")
    from moe_decode_megakernel_02_gb300.latent import LatentPages
    # every row of the one page is the same place (rows are written one a call)
    cache = LatentPages(latent.expand(1, ps, 512), rope.expand(1, ps, 64))
    table = torch.zeros((1, cols), dtype=torch.int32, device="cuda")
    freq = torch.tensor([1e6 / 1.07 ** i for i in range(32)], dtype=torch.float64, device="cuda")
    at = cols * ps - 1
    x = torch.randn((1, 1, 576), device="cuda")
    cache.write(table, ints(at), x, inv_freq=freq)
    want, size = expected(x[:, :, None, 512:], torch.ones((1, 1), device="cuda"), angles(freq, at), "half", 0)
    err = (rope[0, 0].double() - want[0, 0, 0]).abs()
    bound = size[0, 0, 0] * (2.0 ** -21 + at * 2.0 ** -60 * 2 * math.pi) + want[0, 0, 0].abs() * 2.0 ** -11 + 2.0 ** -25
    assert (err <= bound).all()
