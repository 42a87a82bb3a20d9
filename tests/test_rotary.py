"""Rotation by positions, against the definition in 64 bits.

Tolerance. An angle is exact to 2^-25 half turns (pi 2^-25 radians), the sine and cosine to 2 units of the last place
(2^-23), their scaling, two products and a sum to 2^-24 each of what they give: below 2^-21 (|x| + |y|) |magnitude| for a
pair (x, y). The result is rounded once to its type, eps/2 of the value, for fp16 at least half its least step, 2^-25.
"""
import ctypes
import math

import pytest
import torch

import moe_decode_megakernel_02_gb300 as mk
from moe_decode_megakernel_02_gb300 import rotary

gpu = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def expected(x, at, freq, layout, first, magnitude=1.0, inverse=False):
    """x [batch, tokens, heads, head_dim], at [batch, tokens]: (values, the pairs' magnitudes) in 64 bits."""
    n = 2 * freq.shape[0]
    y, size = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    part = y[..., first:first + n].clone()
    a = at.double()[..., None, None] * freq * (-1 if inverse else 1)
    i0 = torch.arange(n // 2) if layout == "half" else torch.arange(0, n, 2)
    i1 = i0 + (n // 2 if layout == "half" else 1)
    u, v = part[..., i0], part[..., i1]
    y[..., first + i0] = magnitude * (u * a.cos() - v * a.sin())
    y[..., first + i1] = magnitude * (u * a.sin() + v * a.cos())
    for i in (i0, i1):
        size[..., first + i] = (u.abs() + v.abs()) * abs(magnitude)
    return y, size


def check(got, want, size):
    step = torch.finfo(got.dtype).eps / 2
    least = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
    err = (got.double() - want).abs()
    assert (err <= size * 2.0 ** -21 + want.abs() * (step + 2.0 ** -21) * (size > 0) + least * (size > 0)).all(), err.max()


# ---------------------------------------------------------------- without a GPU

def _args(**over):
    one = 4096  # aligned, never followed
    r = dict(inv_freq=one, n=64, layout=mk.ROTARY_HALF, magnitude=1.0, inverse=0)
    x = dict(data=one, seq_stride=256, token_stride=256, head_stride=64, dtype=mk.DT_BF16, reserved=0)
    a = dict(positions=one, position_stride=0, batch=2, n_tokens=1, n_heads=4, head_dim=64, first=0, reserved=0)
    o = dict(x)
    for key, val in over.items():
        group, name = key.split("__")
        {"r": r, "x": x, "a": a, "o": o}[group][name] = val
    p = ctypes.pointer
    return mk.RotationStruct(rotary=p(mk.RotaryStruct(**r)), x=p(mk.RowsStruct(**x)), out=p(mk.RowsStruct(**o)), **a)


@pytest.mark.parametrize("over,code", [
    (dict(r__inv_freq=None), mk.ERR_INVALID_ARG), (dict(r__inv_freq=4100), mk.ERR_INVALID_ARG),
    (dict(r__n=0), mk.ERR_INVALID_ARG), (dict(r__n=63), mk.ERR_INVALID_ARG), (dict(r__n=258), mk.ERR_INVALID_ARG),
    (dict(r__layout=2), mk.ERR_INVALID_ARG), (dict(r__magnitude=math.nan), mk.ERR_INVALID_ARG),
    (dict(r__magnitude=math.inf), mk.ERR_INVALID_ARG),
    (dict(a__positions=None), mk.ERR_INVALID_ARG), (dict(a__positions=4098), mk.ERR_INVALID_ARG),
    (dict(x__data=None), mk.ERR_INVALID_ARG), (dict(x__data=4097), mk.ERR_INVALID_ARG),
    (dict(o__data=None), mk.ERR_INVALID_ARG), (dict(o__dtype=mk.DT_F16), mk.ERR_INVALID_ARG),
    (dict(x__dtype=9), mk.ERR_INVALID_ARG), (dict(a__first=-1), mk.ERR_INVALID_ARG),
    (dict(a__first=1), mk.ERR_INVALID_ARG), (dict(a__head_dim=32), mk.ERR_INVALID_ARG),
    (dict(a__batch=-1), mk.ERR_INVALID_ARG), (dict(a__n_tokens=-1), mk.ERR_INVALID_ARG),
    (dict(a__n_heads=-1), mk.ERR_INVALID_ARG), (dict(a__position_stride=-1), mk.ERR_INVALID_ARG),
    (dict(a__batch=1 << 20, a__n_tokens=1 << 10), mk.ERR_UNSUPPORTED), (dict(a__n_heads=5000), mk.ERR_UNSUPPORTED),
    (dict(a__head_dim=1 << 17), mk.ERR_UNSUPPORTED),
    (dict(a__batch=0), mk.OK), (dict(a__n_tokens=0), mk.OK), (dict(a__n_heads=0), mk.OK),
])
def test_refusals(over, code):
    assert mk.lib().mk_rotate(ctypes.byref(_args(**over)), None) == code
    assert mk.lib().mk_rotate(None, None) == mk.ERR_INVALID_ARG


def test_frequencies():
    f = rotary.frequencies(8, theta=100.0, device="cpu")
    assert f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([1.0, 100.0 ** -0.25, 100.0 ** -0.5, 100.0 ** -0.75], dtype=torch.float64))
    assert torch.equal(rotary.frequencies(8, theta=100.0, factor=4.0, device="cpu"), f / 4)
    # within a trained length of 2000 positions: pair 0 turns 318 times and stays, the last one 10 times: in between
    g = rotary.frequencies(8, theta=100.0, factor=4.0, original=2000, device="cpu")
    turns = f * 2000 / (2 * math.pi)
    keep = ((turns - 1) / 31).clamp(0, 1)
    assert torch.allclose(g, f * keep + f / 4 * (1 - keep)) and g[0] == f[0] and f[3] / 4 < g[3] < f[3]
    assert rotary.magnitude(1.0) == 1.0 and abs(rotary.magnitude(8.0) - (0.1 * math.log(8) + 1)) < 1e-15
    for bad in (dict(n=7), dict(n=0), dict(n=8, theta=0.0), dict(n=8, factor=-1.0), dict(n=8, original=0)):
        with pytest.raises(ValueError):
            rotary.frequencies(device="cpu", **bad)


def test_the_binding_refuses_what_is_not_on_a_gpu():
    with pytest.raises(ValueError):
        rotary.rotate(torch.zeros(1, 1, 1, 8), torch.zeros(1, dtype=torch.int32), rotary.frequencies(8, device="cpu"))


# ---------------------------------------------------------------- on the GPU

@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,T,H,D,first,n", [
    (1, 1, 1, 64, 0, 64), (2, 3, 16, 192, 128, 64), (3, 17, 5, 128, 0, 128), (1, 300, 2, 80, 16, 64), (2, 5, 3, 70, 3, 64),
    (1, 2, 1, 2, 0, 2), (4, 1, 40, 256, 0, 256), (1, 9, 7, 50, 1, 46), (2, 1000, 1, 64, 0, 64), (1, 3, 129, 96, 0, 96),
])
def test_against_the_definition(dtype, layout, B, T, H, D, first, n):
    g = torch.Generator(device="cuda").manual_seed(B + T + H + D)
    x = torch.randn((B, T, H, D), generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 8192, (B,), generator=g, device="cuda").to(torch.int32)
    freq = rotary.frequencies(n)
    at = pos[:, None] + torch.arange(T, device="cuda")
    got = rotary.rotate(x, pos, freq, layout=layout, first=first, magnitude=1.25)
    check(got, *expected(x, at, freq, layout, first, 1.25))
    out = torch.empty_like(x)
    assert rotary.rotate(x, at.to(torch.int32).contiguous(), freq, layout=layout, first=first, magnitude=1.25,
                         out=out) is out
    assert torch.equal(out, got)
    # where it is: the same values, the others left alone
    y = x.clone()
    rotary.rotate(y, pos, freq, layout=layout, first=first, magnitude=1.25, out=y)
    assert torch.equal(y, got)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offset", [0, 1])
def test_strides(dtype, offset):
    """The rope part of a fused projection, heads before tokens, aligned and not."""
    g = torch.Generator(device="cuda").manual_seed(5)
    wide = torch.randn((2, 6, 11, 200 + 2 * offset), generator=g, device="cuda").to(dtype)
    x = wide.transpose(1, 2)[..., 128 + offset:192 + offset]  # [2, 11, 6, 64]
    pos = torch.tensor([7, 100000], dtype=torch.int32, device="cuda")
    at = pos[:, None] + torch.arange(11, device="cuda")
    freq = rotary.frequencies(64)
    want = expected(x, at, freq, "half", 0)
    check(rotary.rotate(x, pos, freq), *want)
    kept = wide.clone()
    rotary.rotate(x, pos, freq, out=x)
    check(x, *want)
    kept.transpose(1, 2)[..., 128 + offset:192 + offset] = x
    assert torch.equal(wide, kept)  # nothing else was written


@gpu
@pytest.mark.parametrize("at", [0, 1, -5, 1 << 20, (1 << 31) - 1, -(1 << 31)])
def test_far_positions(at):
    """Angles of 2^31 radians and more: the fraction of a turn is exact."""
    freq = torch.tensor([1.0, 0.731, 1e-3, 6.5, 0.0, 1e-9, -0.25, 3.0e4], dtype=torch.float64, device="cuda")
    x = torch.randn((1, 1, 3, 16), device="cuda")
    pos = torch.tensor([at], dtype=torch.int32, device="cuda")
    # the reference: pos * freq / 2 pi modulo 1 in whole numbers of 2^-80ths
    from fractions import Fraction
    two_pi = Fraction(884279719003555, 281474976710656) + Fraction(4967757600021511, 40564819207303340847894502572032)
    two_pi *= 2  # pi as two 64-bit numbers: 2^-106
    turns = [float((Fraction(f) * at / two_pi) % 1) for f in freq.tolist()]
    a = torch.tensor(turns, dtype=torch.float64, device="cuda") * (2 * math.pi)
    want, size = expected(x, torch.ones((1, 1), device="cuda"), a, "half", 0)
    got = rotary.rotate(x, pos, freq)
    # the frequency itself keeps 2^-52 of its turns a position
    slack = abs(at) * freq.abs().repeat(2) / (2 * math.pi) * 2.0 ** -52 * 2 * math.pi
    err = (got.double() - want).abs()
    assert (err <= size * (2.0 ** -21 + slack) + want.abs() * 2.0 ** -20).all(), err.max()


@gpu
def test_inverse_is_the_transpose():
    x = torch.randn((2, 9, 4, 64), device="cuda")
    pos = torch.tensor([3, 77], dtype=torch.int32, device="cuda")
    freq = rotary.frequencies(64)
    for layout in ("half", "interleaved"):
        y = rotary.rotate(x, pos, freq, layout=layout)
        back = rotary.rotate(y, pos, freq, layout=layout, inverse=True)
        assert (back - x).abs().max() <= 4 * 2.0 ** -21 * x.abs().max() * 2
        # <R x, g> = <x, R' g>: the gradient of a rotation, with a magnitude too
        g = torch.randn_like(x)
        lhs = (rotary.rotate(x, pos, freq, layout=layout, magnitude=1.5).double() * g.double()).sum()
        rhs = (x.double() * rotary.rotate(g, pos, freq, layout=layout, magnitude=1.5, inverse=True).double()).sum()
        size = 1.5 * (x.abs().double() * g.abs().double()).sum() * 2
        assert abs(lhs - rhs) <= size * 2.0 ** -20


@gpu
def test_empty_and_captured():
    freq = rotary.frequencies(64)
    none = torch.zeros((0,), dtype=torch.int32, device="cuda")
    assert rotary.rotate(torch.empty((0, 3, 2, 64), device="cuda"), none, freq).shape == (0, 3, 2, 64)
    pos = torch.tensor([5], dtype=torch.int32, device="cuda")
    assert rotary.rotate(torch.empty((1, 0, 2, 64), device="cuda"), pos, freq).shape == (1, 0, 2, 64)
    x = torch.randn((1, 4, 2, 64), device="cuda")
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    rotary.rotate(x, pos, freq, out=out)
    with torch.cuda.graph(graph):
        rotary.rotate(x, pos, freq, out=out)
    pos.fill_(1234)
    x.normal_()
    graph.replay()
    assert torch.equal(out, rotary.rotate(x, pos, freq))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = rotary.rotate(x, pos, freq, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, out)


@gpu
def test_the_binding_refuses():
    x = torch.zeros((2, 3, 4, 64), device="cuda")
    pos = torch.zeros((2,), dtype=torch.int32, device="cuda")
    freq = rotary.frequencies(64)
    for over in (dict(positions=None), dict(positions=pos.long()), dict(positions=pos[:1]), dict(positions=pos.cpu()),
                 dict(positions=torch.zeros((2, 4), dtype=torch.int32, device="cuda")), dict(inv_freq=freq.float()),
                 dict(inv_freq=freq.cpu()), dict(inv_freq=freq[::2]), dict(layout="other"), dict(out=x.half()),
                 dict(out=x[:1]), dict(out=x[:1].expand(2, -1, -1, -1)), dict(x=x.double()), dict(x=x[0]),
                 dict(first=2.5), dict(magnitude="big"), dict(x=x.transpose(2, 3))):
        with pytest.raises(ValueError):
            rotary.rotate(**{**dict(x=x, positions=pos, inv_freq=freq), **over})
    for over in (dict(first=1), dict(first=-1), dict(inv_freq=rotary.frequencies(130)), dict(magnitude=math.nan)):
        with pytest.raises(mk.MKError):
            rotary.rotate(**{**dict(x=x, positions=pos, inv_freq=freq), **over})
