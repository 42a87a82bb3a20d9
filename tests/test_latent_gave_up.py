"""Attention over latent caches and prompts when a role gives up in the middle of its work: a signal that is left out from each
CTA's fourth tile on (MK_FAULT, set on the host), and a short limit.

A row is then right or it is no number (as for a caller without a status), and the call after it is right."""
import pytest
import torch

import moe_decode_megakernel_02_gb300 as mk
from moe_decode_megakernel_02_gb300 import latent
from test_latent import gpu, ints, make_cache, queries
from test_prompt import make, starts


def check(call, status, monkeypatch, some):
    """some: whether there are rows that are done before."""
    want, wlse = call()
    assert status.item() == mk.OK
    monkeypatch.setenv("MK_WAIT_NS", "3000000")
    monkeypatch.setenv("MK_FAULT", "skip_late_attend_signal")
    for _ in range(5):
        status.zero_()
        out, lse = call()
        assert status.item() == mk.ERR_TIMEOUT
        missing = out.isnan().all(-1)
        assert torch.equal(missing, lse.isnan())
        assert torch.equal(out[~missing], want[~missing]) and torch.equal(lse[~missing], wlse[~missing])
        assert missing.any() and (~missing).any() == some
    monkeypatch.delenv("MK_WAIT_NS")
    monkeypatch.delenv("MK_FAULT")
    status.zero_()
    out, lse = call()
    assert status.item() == mk.OK and torch.equal(out, want) and torch.equal(lse, wlse)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,T,H,L,rank,some", [(1, 1, 16, 40000, 512, False), (3, 7, 16, 9000, 512, False), (400, 1, 16, 60, 512, True),
                                               (400, 1, 40, 60, 512, True), (500, 2, 9, 90, 256, True)])
def test_latents(dtype, B, T, H, L, rank, some, monkeypatch):
    """Pieces that are joined, CTAs of many whole ones (the first ones are done before); 16, 32 and 64 rows a block."""
    cols = -(-L // 64)
    cache = make_cache(dtype, max(cols, 40), 64, rank=rank)
    g = torch.Generator().manual_seed(1)
    table = torch.randint(0, max(cols, 40), (B, cols), generator=g).to(torch.int32).cuda()
    lens = torch.randint(L - 20, L + 1, (B,), generator=g).to(torch.int32).cuda()
    q, qr = queries(dtype, B, T, H, rank=rank)
    status = ints(0)
    check(lambda: cache.attend(table, lens, q, qr, 0.07, return_lse=True, status=status), status, monkeypatch, some)


@gpu
@pytest.mark.parametrize("nq,nk,H,some", [([700, 30], [700, 1500], 2, True), ([100, 20], [1000, 130], 2, True), ([1], [20000], 2, False),
                                          ([256], [9000], 3, False), ([300], [5000], 1, False)])
def test_prompts(nq, nk, H, some, monkeypatch):
    """Blocks of one CTA, and clusters of 2 to 8, whose CTAs hand on rows over what the copies wrote to."""
    q, k, r, v = make(torch.bfloat16, nq, nk, H)
    qa, ka, status = starts(nq), starts(nk), ints(0)
    check(lambda: latent.attend_prompt(q, k, r, v, qa, ka, 0.07, return_lse=True, status=status), status, monkeypatch, some)
