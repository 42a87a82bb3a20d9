"""Rotary positions: mk_rotate (include/mk.h), and the frequencies it takes.

    freq = frequencies(64, theta=1e4, device="cuda")     # float64 [32], radians a position
    q_rope = rotate(q[..., 128:], positions, freq)        # the last 64 values of every head, into a new tensor
    rotate(q, positions, freq, first=128, out=q)          # or where they are

Calls run on the current stream (or `stream`) of x's device and may be captured into a CUDA graph; they record no
gradients (with inverse=True a call is the transpose of the one without).
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import ROTARY_HALF, ROTARY_PAIRS, RotaryStruct, RotationStruct, _check, lib
from .pages import _launch, _rows, _written

_LAYOUT = {"half": ROTARY_HALF, "interleaved": ROTARY_PAIRS}
_ROTARY = struct.Struct("Pii fi")
_ROTATE = struct.Struct("PPqPP iiiiii Pii fi Pqqqii Pqqqii")
_RotateBytes, _RotaryBytes = ctypes.c_char * _ROTATE.size, ctypes.c_char * _ROTARY.size
assert _ROTARY.size == ctypes.sizeof(RotaryStruct) == 24
assert ctypes.sizeof(RotationStruct) == 64 and _ROTATE.size == 64 + 24 + 2 * 40


def frequencies(n, theta=1e4, factor=1.0, original=None, low=1.0, high=32.0, device="cuda"):
    """The n/2 frequencies theta^(-2i/n) of n rotated values, float64 radians a position.

    factor > 1 stretches positions for contexts longer than a model was trained on. Without `original` every
    frequency is divided by it. With it (the trained context's length) a pair that turns more than `high` times within
    that length keeps its frequency, one that turns less than `low` times is divided by factor, and between them the
    share that is kept falls linearly with the number of turns; magnitude(factor) goes with it. Recipes whose
    share falls linearly with the pair's index give other angles between the two: for a model trained with one of them,
    pass frequencies of your own."""
    if n < 2 or n % 2:
        raise ValueError(f"n must be even and at least 2, got {n}")
    if not (theta > 0 and factor > 0):
        raise ValueError(f"theta and factor must be above 0, got {theta} and {factor}")
    f = [theta ** (-2.0 * i / n) for i in range(n // 2)]
    if original is None:
        f = [x / factor for x in f]
    else:
        if not (original > 0 and high > low):
            raise ValueError("original must be above 0, high above low")

        def stretched(x):
            keep = min(1.0, max(0.0, (x * original / (2 * math.pi) - low) / (high - low)))
            return x * keep + x / factor * (1 - keep)

        f = [stretched(x) for x in f]
    return torch.tensor(f, dtype=torch.float64, device=device)


def magnitude(factor):
    """What cosines and sines are scaled by beside stretched frequencies: 0.1 ln(factor) + 1, 1 up to factor 1."""
    return 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0


def _freq(inv_freq, device):
    """The address and number of values of some frequencies."""
    if inv_freq.dtype is not torch.float64 or inv_freq.dim() != 1 or inv_freq.device != device or not inv_freq.is_contiguous():
        raise ValueError(f"inv_freq must be a contiguous float64 tensor [pairs] on {device}, got {inv_freq.dtype} "
                         f"{tuple(inv_freq.shape)} on {inv_freq.device}")
    return inv_freq.data_ptr(), 2 * inv_freq.shape[0]


def _layout(layout):
    code = _LAYOUT.get(layout)
    if code is None:
        raise ValueError(f"layout must be 'half' or 'interleaved', got {layout!r}")
    return code


def rotate(x, positions, inv_freq, layout="half", first=0, magnitude=1.0, inverse=False, out=None, stream=None):
    """Rows x, [batch, tokens, heads, head_dim] (float32, bfloat16 or float16), with values first .. first + n - 1 of
    every head turned by their position's angles, n being twice the number of frequencies.

    positions: int32 [batch], token t of sequence b at positions[b] + t, or int32 [batch, tokens]; inv_freq: float64
    [n / 2], radians a position; layout "half": value i turns with value i + n/2, "interleaved": value 2i with
    2i + 1; magnitude scales the turned values; inverse turns back. Returns `out` (of x's type and shape, x itself
    allowed, no other overlap), a new tensor when not given."""
    if not x.is_cuda:
        raise ValueError(f"x must be a CUDA tensor, got one on {x.device}")
    dev = x.device
    rx = _rows(x, "x", dev)
    shape = x.shape
    if positions is None or positions.dtype is not torch.int32 or positions.device != dev or not positions.is_contiguous() \
            or (positions.shape != shape[:1] and positions.shape != shape[:2]):
        raise ValueError(f"positions must be a contiguous int32 tensor {tuple(shape[:1])} or {tuple(shape[:2])} on {dev}")
    f, n = _freq(inv_freq, dev)
    code = _layout(layout)
    if out is not None:
        if out.dtype is not x.dtype or out.shape != shape:
            raise ValueError(f"out must have x's type and shape, {x.dtype} {tuple(shape)}")
        _written(out, "out")
    return _launch(dev, stream, _rotate, (x, rx, positions, f, n, code, first, magnitude, inverse, out))


def _rotate(h, x, rx, positions, f, n, code, first, mag, inverse, out):
    shape = x.shape
    B, T, H, D = shape
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
        ro = (out.data_ptr(), T * H * D, H * D, D, rx[4], 0)
    else:
        ro = _rows(out, "out", x.device)
    buf = _RotateBytes()
    at = ctypes.addressof(buf)
    try:
        _ROTATE.pack_into(buf, 0, at + 64, positions.data_ptr(), T if positions.dim() == 2 else 0, at + 88,
                          at + 128, B, T, H, D, first, 0, f, n, code, mag, bool(inverse), *rx, *ro)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"first and magnitude must be numbers in range: {e}") from None
    if B and T and H:
        rc = lib().mk_rotate(at, h)
        if rc:
            _check(rc)
    return out
