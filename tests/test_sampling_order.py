"""Sampling: rows that outnumber the device because their slices leave room for one CTA an SM; the largest temperature."""
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


@gpu
@pytest.mark.parametrize("V", [3, 5000])
@pytest.mark.parametrize("top_p", [None, 0.999999])
def test_an_infinite_temperature_gives_every_unmasked_token_the_same_weight(V, top_p):
    """Also where logits lie further apart than the largest number (masks of the type's lowest value)."""
    inf, lowest = float("inf"), torch.finfo(torch.float32).min
    x = torch.full((4, V), lowest, device="cuda")
    x[:, ::2] = 3e38
    x[3] = -inf
    x[3, 1] = lowest
    u = torch.tensor([0.0, 0.5, 0.9999999, 0.7], device="cuda")
    kw = {} if top_p is None else dict(top_p=torch.full((4,), top_p, device="cuda"))
    tok, prob, kept = sampling.sample(x, u, temperature=torch.full((4,), inf, device="cuda"), return_details=True, **kw)
    assert tok[0] == 0 and tok[3] == 1
    if top_p is None:
        assert tok.tolist() == [0, V // 2, V - 1, 1] and kept.tolist() == [V, V, V, 1]
        assert torch.equal(prob, 1 / kept.float())
    else:  # at most the last rank falls away
        assert all(V - 1 <= n <= V for n in kept[:3].tolist())
