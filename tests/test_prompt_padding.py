"""Prompts of a padded batch: most sequences without queries, with and without keys, around few that have some."""
import pytest
import torch

from moe_decode_megakernel_02_gb300 import latent
from test_latent import gpu
from test_prompt import check, make, starts


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("nq,nk,H", [([1] + [0] * 15, [16000] + [0] * 15, 3), ([0] * 300 + [1], [0] * 300 + [9000], 2),
                                     ([0] * 40 + [300] + [0] * 700, [2] * 40 + [300] + [3] * 700, 16),
                                     ([0, 1, 0, 1, 0, 257, 0], [5, 8000, 0, 1, 9, 700, 3000], 5), ([1] * 9 + [0] * 50, [1000] * 9 + [0] * 50, 2),
                                     ([2, 0, 0, 0], [5000, 5000, 0, 1], 1)])
def test_against_the_definition(dtype, nq, nk, H):
    q, k, r, v = make(dtype, nq, nk, H)
    qa, ka = starts(nq), starts(nk)
    out, lse = latent.attend_prompt(q, k, r, v, qa, ka, 0.07, return_lse=True)
    check(q, k, r, v, qa, ka, 0.07, out, lse)
