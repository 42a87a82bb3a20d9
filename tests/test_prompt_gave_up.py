"""Prompts of clusters whose waits run out: no CTA of a cluster takes the others' unfinished rows for numbers."""
import pytest
import torch

from moe_decode_megakernel_02_gb300 import latent
from test_latent import gpu
from test_prompt import make, starts


@gpu
@pytest.mark.parametrize("nq,nk,H", [(256, 9000, 3), (1, 20000, 2), (300, 5000, 1)])
def test_every_row_of_a_clustered_call_that_gave_up_is_no_number(nq, nk, H, monkeypatch):
    """A signal that is left out: the last rows of a block too, whose marks lie where the copied keys did."""
    q, k, r, v = make(torch.bfloat16, [nq], [nk], H)
    at, ka = starts([nq]), starts([nk])
    monkeypatch.setenv("MK_WAIT_NS", "5000000")
    monkeypatch.setenv("MK_FAULT", "skip_attend_signal")
    for _ in range(10):
        out, lse = latent.attend_prompt(q, k, r, v, at, ka, 0.07, return_lse=True)
        assert bool(out.isnan().all()) and bool(lse.isnan().all())
