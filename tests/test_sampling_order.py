"""Sampling where rows outnumber the device because their slices leave room for one CTA an SM."""
import pytest
import torch

from moe_decode_megakernel_02_gb300 import sampling
from test_sampling import gpu, settings


@gpu
@pytest.mark.parametrize("R,V,dtype", [(18, 300000, torch.float32), (37, 340001, torch.float32), (20, 360448, torch.float16)])
def test_rows_of_large_slices_give_what_they_give_alone(R, V, dtype):
    g = torch.Generator(device="cuda").manual_seed(R)
    x = (torch.randn((R, V), generator=g, device="cuda") * 3).to(dtype)
    u = torch.rand((R,), generator=g, device="cuda")
    T, k, p, least = settings(R, g)
    p[:2], k[1], T[1] = torch.tensor([1.0, 0.9], device="cuda"), 0, 1.0  # a costly row behind one that is not
    got = sampling.sample(x, u, temperature=T, top_k=k, top_p=p, min_p=least, return_details=True)
    for r in range(0, R, 4):
        cut = slice(r, r + 4)
        want = sampling.sample(x[cut], u[cut], temperature=T[cut], top_k=k[cut], top_p=p[cut], min_p=least[cut],
                               return_details=True)
        assert all(torch.equal(a[cut], b) for a, b in zip(got, want))
