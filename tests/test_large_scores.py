"""Scores whose own steps are larger than 1: the largest one takes all, equal ones share, and nothing overflows.

Scores here are a scale times sums that are exact in 32 bits and differ by 1 or more; times a scale of 10^6 on their weights are
0 or equal, whatever a 32-bit product of 10^30 loses. An output is then one value, or the mean of four, rounded once."""
import math

import pytest
import torch

from moe_decode_megakernel_02_gb300 import latent
from test_latent import gpu, ints

TYPES = [torch.bfloat16, torch.float16]
SCALES = [1.1e6, 1.3e7, 1e8, 7.7e8, 1e10, 3e14, 1e20, 9e27, -1e7, -1e9, -2e25]


def inputs(dtype, n, width, sign, seed):
    """[n] scores (whole numbers as two parts, both exact in either type), [n, width] values; the four best are far apart."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randperm(n, generator=g, device="cuda").float()
    x[[5, n // 3, n // 2 + 77, n - 2]] = n + 3.0
    x = sign * x
    high = (x / 128).floor() * 128
    v = torch.randn((n, width), generator=g, device="cuda").to(dtype)
    return x, high.to(dtype), (x - high).to(dtype), v


def check(out, lse, x, v, scale, rows):
    best = (x * (1 if scale > 0 else -1)).double()
    at = (best == best.max()).nonzero().flatten()
    want = v[at].double().mean(0)
    half = torch.finfo(out.dtype).eps / 2
    # (four equal weights: exact; their products' sum and quotient lose less than 2^-20 of the values)
    bound = v[at].double().abs().mean(0) * 2.0 ** -20 + want.abs() * half + (2.0 ** -25 if out.dtype == torch.float16 else 0)
    assert ((out.double() - want).abs() <= bound).all(), (out.double() - want).abs().max()
    z = best.max().item() * abs(scale) + math.log(len(at))
    # (a product of three 32-bit roundings and a last one)
    assert ((lse.double() - z).abs() <= abs(z) * 2.0 ** -21).all()


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("n,H,N", [(300, 1, 1), (4000, 2, 1), (2000, 3, 200)])
def test_prompts(dtype, scale, n, H, N):
    x, high, low, v = inputs(dtype, n, 128, 1 if scale > 0 else -1, n)
    q = torch.zeros((N, H, 192), dtype=dtype, device="cuda")
    q[..., 3] = q[..., 130] = 1
    k = torch.zeros((n, H, 128), dtype=dtype, device="cuda")
    r = torch.zeros((n, 64), dtype=dtype, device="cuda")
    k[..., 3], r[:, 2] = high[:, None], low
    out, lse = latent.attend_prompt(q, k, r, v[:, None].expand(-1, H, -1), ints(0, N), ints(0, n), scale, return_lse=True)
    for i in sorted({0, N - 1, N // 2}):
        m = n - N + i + 1
        check(out[i], lse[i], x[:m], v[:m], scale, H)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("n,T,H,ps", [(300, 1, 16, 64), (4000, 1, 5, 64), (2000, 5, 8, 64), (500, 2, 3, 4)])
def test_absorbed(dtype, scale, n, T, H, ps):
    x, high, low, v = inputs(dtype, n, 512, 1 if scale > 0 else -1, n)
    pages = -(-n // ps)
    cache = latent.LatentPages(torch.zeros((pages, ps, 512), dtype=dtype, device="cuda"), torch.zeros((pages, ps, 64), dtype=dtype, device="cuda"))
    cache.latent.view(-1, 512)[:n] = v
    cache.rope.view(-1, 64)[:n, 2], cache.rope.view(-1, 64)[:n, 9] = high, low
    q = torch.zeros((1, T, H, 512), dtype=dtype, device="cuda")
    qr = torch.zeros((1, T, H, 64), dtype=dtype, device="cuda")
    qr[..., 2] = qr[..., 9] = 1
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    out, lse = cache.attend(table, ints(n), q, qr, scale, return_lse=True)
    for t in range(T):
        m = n - T + t + 1
        check(out[0, t], lse[0, t], x[:m], v[:m], scale, H)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("form", ["prompt", "absorbed"])
def test_scores_a_step_apart(dtype, form):
    """Maxima that rise by one step of a 32-bit score, 4 to 64 powers of 2, from tile to tile: outputs lie between the values."""
    n = 640
    lift = (torch.arange(n, device="cuda") // 32).float() / 8
    v = torch.rand((n, 512), device="cuda").to(dtype) + 1
    for power in (24, 25, 26, 27, 28, 29, 30):
        for part in (0.96, 1.0, 1.03, 1.37, 1.99):
            scale = part * 2.0 ** (power - 20) * math.log(2)
            if form == "prompt":
                q = torch.zeros((1, 1, 192), dtype=dtype, device="cuda")
                q[..., 0], q[..., 128] = 1024, 1
                k, r = torch.zeros((n, 1, 128), dtype=dtype, device="cuda"), torch.zeros((n, 64), dtype=dtype, device="cuda")
                k[..., 0], r[:, 0] = 1024, lift
                out = latent.attend_prompt(q, k, r, v[:, None, :128], ints(0, 1), ints(0, n), scale)
            else:
                cache = latent.LatentPages(v.view(10, 64, 512).contiguous(), torch.zeros((10, 64, 64), dtype=dtype, device="cuda"))
                cache.rope.view(n, 64)[:, 0], cache.rope.view(n, 64)[:, 1] = 1024, lift
                q, qr = torch.zeros((1, 1, 1, 512), dtype=dtype, device="cuda"), torch.zeros((1, 1, 1, 64), dtype=dtype, device="cuda")
                qr[..., 0], qr[..., 1] = 1024, 1
                out = cache.attend(torch.arange(10, dtype=torch.int32, device="cuda")[None], ints(n), q, qr, scale)
            assert ((out >= 1) & (out <= 2)).all(), (power, part, out.min(), out.max())
