"""Rows of large and small magnitudes into a latent cache: their squares' sum stays in the range of 32 bits."""
import pytest
import torch

from test_latent import ints, make_cache, make_table


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rank", [256, 512, 1024])
@pytest.mark.parametrize("rows,power", [(torch.float32, 59.9), (torch.bfloat16, 59.0), (torch.float32, 40.0), (torch.float32, -50.0)])
def test_magnitudes(dtype, rank, rows, power):
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((1, 5, rank + 64), generator=g, device="cuda").clamp(-1, 1)
    x[:, 1, :rank] = 1
    x = (x * 2.0 ** power).to(rows)
    x[..., rank:] = 0
    cache = make_cache(dtype, 1, 8, rank=rank)
    eps = 0.0 if power < 0 else 1e-6
    cache.write(make_table(1, 1, 1), ints(0), x, gain=torch.ones((rank,), device="cuda"), eps=eps)
    c = x[0, :, :rank].double()
    want = c / (c.square().mean(-1, keepdim=True) + eps).sqrt()
    half = torch.finfo(dtype).eps / 2
    assert ((cache.latent[0, :5].double() - want).abs() <= want.abs() * (half + 2.0 ** -18) + (2.0 ** -25 if dtype == torch.float16 else 0)).all()
