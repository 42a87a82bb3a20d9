"""Weights far below the largest one in fp16: many of them together count.

One position takes nearly all and has a value of 0, many take some 2^-27 of it each and have values of 1, so that the output
is their share. Tolerance, as in test_latent, but what a weight loses to fp16 is at least 2^-32 of the largest one (not
2^-25): scores here are exact; a 32-bit exponential, the sums and the pieces' join lose less than 2^-18 of the output, a
weight half a step of fp16 or 2^-32, the output half a step or 2^-25.
"""
import math

import pytest
import torch

from moe_decode_megakernel_02_gb300 import latent
from test_latent import ints

gpu = pytest.mark.gpu
LOW = -18.5  # e^LOW is 2^-26.7


def close(out, lse, n):
    w = math.exp(LOW)
    want = n * w / (1 + n * w)
    sums = 2.0 ** -15 + 2.0 ** -18
    bound = n * 2.0 ** -32 + want * (2.0 ** -11 + 2.0 ** -13 + sums) + want * 2.0 ** -11 + 2.0 ** -25
    assert (out.double() - want).abs().max() <= bound, (out.double().min().item(), out.double().max().item(), want)
    assert (lse.double() - math.log1p(n * w)).abs().max() <= sums


@gpu
@pytest.mark.parametrize("first", [True, False])
def test_prompts(first):
    n, H = 65535, 160  # (as many heads as do not share their keys out)
    r = torch.zeros((n + 1, 64), dtype=torch.float16, device="cuda")
    v = torch.ones((n + 1, 1, 128), dtype=torch.float16, device="cuda")
    top = 0 if first else n
    r[:, 0] = LOW
    r[top], v[top] = 0, 0
    q = torch.zeros((1, H, 192), dtype=torch.float16, device="cuda")
    q[..., 128] = 1
    k = torch.zeros((n + 1, 1, 128), dtype=torch.float16, device="cuda").expand(-1, H, -1)
    out, lse = latent.attend_prompt(q, k, r, v.expand(-1, H, -1), ints(0, 1), ints(0, n + 1), 1.0, return_lse=True)
    close(out, lse, n)


@gpu
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("T,H", [(1, 16), (7, 16)])
def test_absorbed(first, T, H):
    """As many sequences (of the same pages) as give a CTA a few each; all tokens see nearly all of it."""
    n, ps, B = 16384, 64, 304
    cache = latent.LatentPages(torch.ones((n // ps, ps, 512), dtype=torch.float16, device="cuda"),
                               torch.zeros((n // ps, ps, 64), dtype=torch.float16, device="cuda"))
    top = 0 if first else n - T
    cache.rope[..., 0] = LOW
    cache.rope[top // ps, top % ps], cache.latent[top // ps, top % ps] = 0, 0
    table = torch.arange(n // ps, dtype=torch.int32, device="cuda").expand(B, -1)
    q = torch.zeros((B, T, H, 512), dtype=torch.float16, device="cuda")
    qr = torch.zeros((B, T, H, 64), dtype=torch.float16, device="cuda")
    qr[..., 0] = 1
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    out, lse = cache.attend(table, lens, q, qr, 1.0, return_lse=True)
    for t in range(T):
        close(out[:, t], lse[:, t], n - T + t)


@gpu
def test_weights_that_rise_slowly_stay_in_range():
    """A score that rises less than 2^8 a tile does not move the reference: such weights are the largest that occur."""
    n = 4096
    step = 5.4  # of e: 2^7.8 a tile of 128 keys, and twice so before the reference moves
    j = torch.arange(n, device="cuda")
    r = torch.zeros((n, 64), dtype=torch.float16, device="cuda")
    r[:, 0] = ((j // 128) * step).half()
    v = torch.randn((n, 1, 128), device="cuda").half()
    q = torch.zeros((1, 1, 192), dtype=torch.float16, device="cuda")
    q[..., 128] = 1
    k = torch.zeros((n, 1, 128), dtype=torch.float16, device="cuda")
    out, lse = latent.attend_prompt(q, k, r, v, ints(0, 1), ints(0, n), 1.0, return_lse=True)
    x = r[:, 0].double()
    w = torch.softmax(x, 0)
    want = w @ v[:, 0].double()
    bound = (w @ v[:, 0].double().abs()) * (2.0 ** -11 + 2.0 ** -17) + want.abs() * 2.0 ** -11 + 2.0 ** -25
    assert ((out[0, 0].double() - want).abs() <= bound).all()
    assert abs(lse.item() - torch.logsumexp(x, 0).item()) <= 2.0 ** -18 + 200 * 2.0 ** -22
