"""Forms of the latent operators' kernels that other tests do not reach: 17 to 32 rows a block and many rows of rank 256, pages
too small for tensor maps there, wide rope parts beside short latents and the other way round, rows off 16 bytes."""
import pytest
import torch

from moe_decode_megakernel_02_gb300 import rotary
from test_latent import check_attend, ints, make_cache, make_table, queries
from test_rotary import expected as turned

gpu = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rank", [256, 512])
@pytest.mark.parametrize("T,H", [(2, 16), (3, 6), (1, 17), (1, 32), (4, 12), (1, 33)])
def test_rows_of_a_block(dtype, rank, T, H):
    cache = make_cache(dtype, 90, 32, rank=rank)
    table = make_table(3, 30, 90)
    q, qr = queries(dtype, 3, T, H, rank=rank)
    check_attend(cache, table, ints(30 * 32, 203, 2), q, qr, 0.07, starts=ints(0, 37, 0))


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rank", [256, 512])
@pytest.mark.parametrize("T,H", [(1, 16), (2, 9), (3, 16)])
def test_many_rows(dtype, rank, T, H):
    """More rows than four an SM, whose tiles lie in two or three CTAs' stretches."""
    B, ps = 64, 64
    cache = make_cache(dtype, 300, ps, rank=rank)
    table = torch.randint(0, 300, (B, 18), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    lens = torch.randint(600, 18 * ps + 1, (B,), generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    lens[5] = 0
    q, qr = queries(dtype, B, T, H, rank=rank)
    check_attend(cache, table, lens, q, qr, 0.07)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ps", [1, 4])
def test_small_pages_of_rank_256(dtype, ps):
    cache = make_cache(dtype, 200, ps, rank=256)
    table = make_table(2, 60, 200)
    q, qr = queries(dtype, 2, 2, 5, rank=256)
    check_attend(cache, table, ints(60 * ps, 17), q, qr, 0.07, starts=ints(3, 0))


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("rank,rope,layout", [(512, 128, "half"), (256, 256, "interleaved"), (1024, 64, "half"), (520, 8, "interleaved"),
                                              (1024, 72, "half"), (512, 64, "interleaved")])
def test_writes(dtype, rows, offset, rank, rope, layout):
    B, T, ps = 2, 21, 16
    g = torch.Generator(device="cuda").manual_seed(rank + rope)
    cache = make_cache(dtype, 8, ps, rank, rope)
    table = make_table(B, 4, 8)
    wide = (torch.randn((B, T, rank + rope + 8), generator=g, device="cuda") * 3).to(rows)
    x = wide[..., offset:offset + rank + rope]
    gain = 1 + 0.2 * torch.randn((rank,), generator=g, device="cuda")
    freq, pos = rotary.frequencies(rope), ints(0, 40)
    cache.write(table, pos, x, gain=gain, inv_freq=freq, layout=layout, magnitude=1.25)
    half = torch.finfo(dtype).eps / 2
    least = 2.0 ** -25 if dtype == torch.float16 else 0.0
    for b in range(B):
        at = pos[b] + torch.arange(T, device="cuda")
        page, row = table[b, at // ps].long(), at % ps
        c = x[b, :, :rank].double()
        c = c / (c.square().mean(-1, keepdim=True) + 1e-6).sqrt() * gain.double()
        assert ((cache.latent[page, row].double() - c).abs() <= c.abs() * (half + 2.0 ** -18) + least).all()
        r, size = turned(x[None, b, :, None, rank:], at[None], freq, layout, 0, 1.25)
        r, size = r[0, :, 0], size[0, :, 0]
        assert ((cache.rope[page, row].double() - r).abs() <= size * 2.0 ** -21 + r.abs() * (half + 2.0 ** -21) + least).all()
