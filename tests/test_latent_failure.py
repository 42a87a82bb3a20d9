"""Latent attention and prompts when a wait inside a kernel runs out: a signal that is left out on purpose (MK_FAULT, set on
the host), a short limit, and the call after it. Nothing faults: every role of the kernel gives up and the CTA leaves."""
import pytest
import torch

import moe_decode_megakernel_02_gb300 as mk
from moe_decode_megakernel_02_gb300 import latent
from test_latent import gpu, ints, make_cache, make_table, queries
from test_prompt import make, starts


def a_call(kind):
    """Fewer tiles a CTA than its ring holds (all copies are under way when the wait runs out), and more; several pieces."""
    if kind.startswith("prompt"):
        nq, nk = ([100], [100]) if kind == "prompt short" else ([700, 30], [900, 4000])
        q, k, r, v = make(torch.bfloat16, nq, nk, 2)
        return lambda status=None: latent.attend_prompt(q, k, r, v, starts(nq), starts(nk), 0.07, return_lse=True, status=status)
    B, T, lens = {"short": (1, 1, [100]), "long": (2, 1, [40000, 30000]), "rows": (3, 7, [3000, 500, 2000])}[kind]
    cols = -(-max(lens) // 64)
    cache = make_cache(torch.bfloat16, B * cols, 64)
    table, n = make_table(B, cols, B * cols), ints(*lens)
    q, qr = queries(torch.bfloat16, B, T, 16)
    return lambda status=None: cache.attend(table, n, q, qr, 0.07, return_lse=True, status=status)


KINDS = ["short", "long", "rows", "prompt short", "prompt long"]


@gpu
@pytest.mark.parametrize("kind", KINDS)
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(kind, monkeypatch):
    call = a_call(kind)
    status = ints(0)
    want, wlse = call(status)
    assert int(status) == 0
    monkeypatch.setenv("MK_WAIT_NS", "20000000")
    monkeypatch.setenv("MK_FAULT", "skip_attend_signal")
    call(status)
    assert int(status) == mk.ERR_TIMEOUT
    monkeypatch.delenv("MK_FAULT")
    monkeypatch.delenv("MK_WAIT_NS")
    status.zero_()
    out, lse = call(status)
    assert int(status) == 0 and torch.equal(out, want) and torch.equal(lse, wlse)


@gpu
@pytest.mark.parametrize("kind", KINDS)
def test_what_a_call_that_gave_up_leaves_is_no_number(kind, monkeypatch):
    """A caller without a status sees it in the output."""
    call = a_call(kind)
    monkeypatch.setenv("MK_WAIT_NS", "20000000")
    monkeypatch.setenv("MK_FAULT", "skip_attend_signal")
    out, lse = call()
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())
