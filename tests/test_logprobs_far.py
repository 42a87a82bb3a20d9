"""Logits so far apart that their difference is beyond 32 bits, at temperatures that bring them together again.

Tolerance as in test_logprobs."""
import math

import pytest
import torch

from moe_decode_megakernel_02_gb300 import sampling
from test_logprobs import expected

gpu = pytest.mark.gpu


def rows(V, dtype):
    x = torch.tensor([3e38, -3e38, 1e38, 0.0, -2.5e38, 3.3e38, -3.3e38], device="cuda").repeat(V // 7 + 1)[:V].to(dtype)
    return x.repeat(4, 1)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [7, 5003, 40000])
@pytest.mark.parametrize("top", [0, 5])
def test_far_logits(dtype, V, top):
    x = rows(V, dtype)
    x[3, 1::7] = -math.inf
    x[1] = x[1].flip(0)  # (the largest last: every sum so far is taken over)
    T = torch.tensor([1e38, 3e38, math.inf, 2e38], device="cuda")
    tokens = torch.arange(7, dtype=torch.int32, device="cuda").repeat(4, 1)
    got, h, ids, best = sampling.logprobs(x, tokens, top=top, temperature=T)
    logp, entropy, spread = expected(x.double().masked_fill(torch.isinf(T)[:, None] & torch.isfinite(x), 0.0),
                                     T.nan_to_num(1.0, 1.0, 1.0))
    base = (V / 256 + 32) * 2.0 ** -24 + 2.0 ** -21 * (1 + spread)
    want = logp.gather(1, tokens.long())
    masked = want == -math.inf
    assert torch.equal(got == -math.inf, masked)
    err = (got.double() - want).abs().masked_fill(masked, 0)
    assert (err <= base[:, None] + want.abs() * 2.0 ** -21).all(), err
    assert ((h.double() - entropy).abs() <= base * (1 + spread) * 2).all()
    if top:
        order = x.float().sort(dim=-1, descending=True, stable=True).indices[:, :top]
        assert torch.equal(ids.long(), order)
        want = logp.gather(1, order)
        assert ((best.double() - want).abs() <= base[:, None] + want.abs() * 2.0 ** -21).all()
