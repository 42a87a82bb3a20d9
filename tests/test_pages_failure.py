"""Attention over pages when a wait inside a kernel runs out: a signal that is left out on purpose (MK_FAULT, set on the
host), a short limit, and the call after it. Nothing faults: every role of the kernel gives up and the CTA leaves."""
import pytest
import torch

import moe_decode_megakernel_02_gb300 as mk
from test_pages import FORMATS, build, gpu, ints, widen


def a_call(kind, fmt):
    """Fewer tiles a CTA than its ring holds (all loads are under way when the wait runs out), and more; wide calls."""
    if kind == "wide":
        B, T, Hq, H, ps, shared, lens = 3, 10, 16, 4, 64, 0, [2000, 500, 700]
    else:
        B, T, Hq, H, ps, shared = 20, 1, 64, 8, 64, 128 if kind == "short" else 16384
        lens = [shared + 5 * b + 1 for b in range(B)]
    cache, table, n, q = build(fmt, torch.bfloat16, B, T, Hq, H, 128, ps, lens, shared=shared)
    if kind == "wide":
        table = widen(table, Hq, H, T, ps)
    return cache, lambda status=None: cache.attend(table, n, q, shared_len=shared, return_lse=True, status=status)


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", ["short", "long", "wide"])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(fmt, kind, monkeypatch):
    cache, call = a_call(kind, fmt)
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
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", ["short", "long", "wide"])
def test_what_a_call_that_gave_up_leaves_is_no_number(fmt, kind, monkeypatch):
    """A caller without a status sees it in the output: every row that the launch has a part in is NaN."""
    cache, call = a_call(kind, fmt)
    monkeypatch.setenv("MK_WAIT_NS", "20000000")
    monkeypatch.setenv("MK_FAULT", "skip_attend_signal")
    out, lse = call()
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())
