"""The bindings of the latent operators: what they keep between calls."""
import pytest
import torch

from moe_decode_megakernel_02_gb300 import latent
from test_latent import ints, make_cache, queries

gpu = pytest.mark.gpu


@gpu
def test_what_is_kept_of_shapes_is_bounded():
    """A server's block table grows with its contexts: calls of ever other shapes keep no more than some hundred sizes."""
    cache = make_cache(torch.bfloat16, 1, 64)
    q, qr = queries(torch.bfloat16, 1, 1, 1)
    table, lens = torch.zeros((1, 700), dtype=torch.int32, device="cuda"), ints(64)
    want = cache.attend(table[:, :1], lens, q, qr, 0.1)
    for cols in range(1, 700):
        got = cache.attend(table[:, :cols], lens, q, qr, 0.1)
    assert torch.equal(got, want)
    assert len(latent._NEED) <= 256
