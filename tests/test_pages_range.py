"""Attention over pages at the ends of its values' range: scales, caps and infinities.

The references are those of test_pages.py, in 64 bits. A score's products are summed in 32 bits, at most about
(D + 8) 2^-24 of sum |q k| scale off; the cap's error is relative to the capped score. For |z| >= 1/2, z the score over
the cap, tanh z = 1 - 2 / (e^2z + 1): the exponent's roundings (3 2^-24 of z, times sech^2 z, at most 0.67 2^-23 of 1),
the exponential's 2^-22 (0.79 2^-23), the reciprocal's 2^-23 of at most 0.27, twice (0.54 2^-23), and the roundings of
the sums (0.77 2^-23) make 2.8 2^-23 of the cap, 6 2^-23 of a tanh that is at least 0.46; below, a polynomial and its
7 roundings stay under 2^-20 as well, which the bounds here take with the cap's own two roundings.
"""
import ctypes
import math

import pytest
import torch

import moe_decode_megakernel_02_gb300 as mk
import test_pages as tp
from test_pages import FORMATS, build, gpu, reference, widen


def close(cache, table, lens, q, out, lse, scale, dv, rel=0.0, **kw):
    """Against 64 bits: rel is the cap's error, of a score's size; dv an absolute error of outputs."""
    ref, rlse, mag, reach = reference(cache, table, lens, q, scale, **kw)
    D, cap = q.shape[-1], kw.get("softcap", 0.0)
    far = float(kw["slopes"].abs().max()) * float(lens.max()) if kw.get("slopes") is not None else 0.0
    dx = (D + 8) * 2.0 ** -24 * (reach + far + 1) + rel * (reach.clamp(max=cap) if cap else 0.0) + 2.0 ** -20
    weight = 2 * dx + (2.0 ** -16 if cache.k.dtype == torch.bfloat16 else 2.0 ** -11)
    eps = torch.finfo(q.dtype).eps / 2
    bound = weight[..., None] * mag + eps * (ref.abs() + weight[..., None] * mag) + dv
    d = (out.double() - ref).abs()
    assert bool((d <= bound).all()), f"off by {float((d / bound).max()):.3g} of the bound"
    seen = rlse > -math.inf
    assert bool(((lse.double() - rlse).abs()[seen] <= (dx + 2.0 ** -22 * rlse.abs())[seen]).all())


# what a call's shape leads to: one launch, pieces and a join, 64- and 128-row blocks, whole tiles apart
SHAPES = {"cluster": (2, 3, 4, 2, 64, 16, [70, 41]), "pieces": (8, 3, 8, 2, 128, 64, [3000 + 61 * i for i in range(8)]),
          "wide_heads": (2, 3, 4, 2, 256, 32, [500, 77]), "blocks": (2, 20, 6, 2, 128, 16, [300, 97]),
          "blocks64": (1, 20, 6, 2, 256, 16, [300]), "wide": (3, 10, 16, 4, 128, 16, [2000, 333, 700])}


def shape_of(kind, fmt, qdtype):
    B, T, Hq, H, D, ps, lens = SHAPES[kind]
    cache, table, n, q = build(fmt, qdtype, B, T, Hq, H, D, ps, lens)
    return cache, (widen(table, Hq, H, T, ps) if kind == "wide" else table), n, q, lens, ps


@gpu
@pytest.mark.parametrize("fmt", FORMATS[1:])
@pytest.mark.parametrize("kind", SHAPES)
@pytest.mark.parametrize("qdtype", [torch.bfloat16, torch.float16])
def test_scales_of_either_sign(fmt, kind, qdtype):
    """A value is code x scale, whatever the scale's sign."""
    cache, table, n, q, lens, ps = shape_of(kind, fmt, qdtype)
    cache.v_scale.neg_()
    cache.k_scale[..., ::2].neg_()
    for step in (0, 3):  # all of them negative; two in three
        if step:
            cache.v_scale[..., ::step].abs_()
        out, lse = cache.attend(table, n, q, return_lse=True)
        dv = max(lens) * 2.0 ** -39 * tp.QMAX[fmt] * float(cache.v_scale.abs().max())
        close(cache, table, n, q, out, lse, 1 / math.sqrt(q.shape[-1]), dv + 2.0 ** -24)


@gpu
@pytest.mark.parametrize("fmt", FORMATS[1:])
@pytest.mark.parametrize("kind", SHAPES)
@pytest.mark.parametrize("scale", [math.inf, -math.inf, 1e30, 2.0 ** 40, math.nan])
def test_the_scale_of_a_position_that_is_not_seen_changes_nothing(fmt, kind, scale):
    """Only the last token sees the last position: the others' outputs stay, bit for bit, whatever its V scale."""
    for qdtype in (torch.bfloat16, torch.float16):
        cache, table, n, q, lens, ps = shape_of(kind, fmt, qdtype)
        clean, clse = cache.attend(table, n, q, return_lse=True)
        for b, L in enumerate(lens):
            cache.v_scale[int(table[b, (L - 1) // ps]), :, (L - 1) % ps] = scale
        out, lse = cache.attend(table, n, q, return_lse=True)
        assert torch.equal(out[:, :-1], clean[:, :-1]) and torch.equal(lse, clse)
        if not math.isfinite(scale):
            assert not bool(torch.isfinite(out[:, -1]).any())
        elif qdtype == torch.bfloat16:  # the last token sees it: its error is of that scale
            dv = max(lens) * 2.0 ** -39 * tp.QMAX[fmt] * scale
            close(cache, table, n, q[:, -1:], out[:, -1:], lse[:, -1:], 1 / math.sqrt(q.shape[-1]), dv)


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", list(SHAPES) + ["shared"])
@pytest.mark.parametrize("cap", [3.0, 50.0, 1e3, 1e5, 1e8, 1e30])
def test_caps_of_any_size(fmt, kind, cap):
    """Scores up to some 30, far below and far above the cap: the error is of the score's size, not of the cap's."""
    shared = 0
    if kind == "shared":
        B, T, Hq, H, D, ps, shared = 20, 1, 8, 2, 128, 16, 320
        lens = [shared + 3 + 5 * b for b in range(B)]
        cache, table, n, q = build(fmt, torch.bfloat16, B, T, Hq, H, D, ps, lens, shared=shared)
    else:
        cache, table, n, q, lens, ps = shape_of(kind, fmt, torch.bfloat16)
    D = q.shape[-1]
    for scale, slopes in ((3 / math.sqrt(D), None), (0.02 / math.sqrt(D), torch.full((q.shape[2],), 0.01, device="cuda"))):
        kw = dict(softcap=cap, slopes=slopes)
        out, lse = cache.attend(table, n, q, scale=scale, shared_len=shared, return_lse=True, **kw)
        dv = 2.0 ** -24 if fmt == torch.bfloat16 else max(lens) * 2.0 ** -39 * tp.QMAX[fmt] * float(cache.v_scale.max())
        close(cache, table, n, q, out, lse, scale, dv, rel=2.0 ** -20, **kw)


@pytest.mark.parametrize("cap", [1e-31, 1e31, -1.0, math.nan, math.inf])
def test_caps_out_of_range_are_refused(cap):
    p, t, r, a = tp._structs(a__softcap=cap)
    att = mk.AttentionStruct(pages=ctypes.pointer(p), table=ctypes.pointer(t), q=ctypes.pointer(r), out=ctypes.pointer(r),
                             **a)
    n = ctypes.c_int64()
    assert mk.lib().mk_pages_attend_workspace(ctypes.byref(att), ctypes.byref(n)) == mk.ERR_INVALID_ARG


@gpu
@pytest.mark.parametrize("kind", list(SHAPES) + ["shared"])
@pytest.mark.parametrize("qdtype", [torch.bfloat16, torch.float16])
def test_infinite_values_in_whole_tiles_stay_infinite(kind, qdtype):
    """Positions that every token sees, in tiles without a mask: an infinity times a weight is that infinity."""
    shared = 0
    if kind == "shared":
        B, T, Hq, H, D, ps, shared = 20, 1, 8, 2, 128, 16, 320
        lens = [shared + 3 + 5 * b for b in range(B)]
        cache, table, n, q = build(torch.bfloat16, qdtype, B, T, Hq, H, D, ps, lens, shared=shared)
    else:
        cache, table, n, q, lens, ps = shape_of(kind, torch.bfloat16, qdtype)
    for b, L in enumerate(lens):
        for j, d, x in ((0, 5, math.inf), (1, 9, -math.inf), (17, 11, math.inf), (3, 11, -math.inf), (16, 33, math.inf)):
            cache.v[int(table[b, j // ps]), :, j % ps, d] = x
    out, lse = cache.attend(table, n, q, shared_len=shared, return_lse=True)
    assert bool((out[..., 5] == math.inf).all()) and bool((out[..., 33] == math.inf).all())
    assert bool((out[..., 9] == -math.inf).all()) and bool(torch.isnan(out[..., 11]).all())
    rest = torch.ones(q.shape[-1], dtype=torch.bool, device="cuda")
    rest[[5, 9, 11, 33]] = False
    assert bool(torch.isfinite(out[..., rest]).all()) and bool(torch.isfinite(lse).all())
