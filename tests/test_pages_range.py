"""Attention over pages at the ends of its values' range: scales, caps and infinities.

The references are those of test_pages.py, in 64 bits.
"""
import math

import pytest
import torch

import test_pages as tp
from test_pages import FORMATS, build, gpu, reference, widen


def close(cache, table, lens, q, out, lse, scale, dv, **kw):
    """Against 64 bits: dv is an absolute error of outputs."""
    ref, rlse, mag, reach = reference(cache, table, lens, q, scale, **kw)
    D = q.shape[-1]
    far = float(kw["slopes"].abs().max()) * float(lens.max()) if kw.get("slopes") is not None else 0.0
    dx = (D + 8) * 2.0 ** -24 * (reach + far + 1) + 2.0 ** -20
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
