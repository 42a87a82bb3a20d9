"""Prompts whose waits run out while copies and products are under way: a limit so short that a role gives up in the middle.

Whenever that is, a row is right or it is no number, as for a caller without a status, and the call after it is right."""
import pytest
import torch

import moe_decode_megakernel_02_gb300 as mk
from moe_decode_megakernel_02_gb300 import latent
from test_latent import gpu, ints
from test_prompt import make, starts


@gpu
@pytest.mark.parametrize("nq,nk,H", [([100], [100], 2), ([700, 30], [900, 4000], 2), ([1], [20000], 2), ([256], [9000], 3), ([300], [5000], 1)])
def test_a_row_is_right_or_no_number(nq, nk, H, monkeypatch):
    """Blocks of one CTA, and clusters of 2, 4 and 8, whose CTAs hand their rows on over what the copies write to."""
    q, k, r, v = make(torch.bfloat16, nq, nk, H)
    qa, ka, status = starts(nq), starts(nk), ints(0)

    def call():
        return latent.attend_prompt(q, k, r, v, qa, ka, 0.07, return_lse=True, status=status)

    want, wlse = call()
    for ns in (1, 1000, 2000, 4000, 6000, 8000, 12000, 20000, 50000, 200000):
        monkeypatch.setenv("MK_WAIT_NS", str(ns))
        for _ in range(20):
            status.zero_()
            out, lse = call()
            wrong, missing = (out != want).any(-1), out.isnan().all(-1)
            assert not (wrong & ~missing).any() and not ((lse != wlse) & ~lse.isnan()).any()
            assert status.item() == (mk.ERR_TIMEOUT if wrong.any() else status.item()) and status.item() in (mk.OK, mk.ERR_TIMEOUT)
    monkeypatch.delenv("MK_WAIT_NS")
    status.zero_()
    out, lse = call()
    assert status.item() == mk.OK and torch.equal(out, want) and torch.equal(lse, wlse)


@gpu
def test_every_row_of_a_clustered_call_that_gave_up_is_no_number(monkeypatch):
    """A signal that is left out: the last rows of a block too, whose marks lie where the copied keys did."""
    q, k, r, v = make(torch.bfloat16, [256], [9000], 3)
    at, ka = starts([256]), starts([9000])
    monkeypatch.setenv("MK_WAIT_NS", "5000000")
    monkeypatch.setenv("MK_FAULT", "skip_attend_signal")
    for _ in range(10):
        out, lse = latent.attend_prompt(q, k, r, v, at, ka, 0.07, return_lse=True)
        assert bool(out.isnan().all()) and bool(lse.isnan().all())
