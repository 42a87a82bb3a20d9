"""Paged KV caches of the caller: rows in (quantised on the way), rows out, and attention over the pages.

Binding of mk_pages_write, mk_pages_read and mk_pages_attend (include/mk.h).
The cache, its block table and everything else are the caller's own tensors;
a `Pages` only describes them. Calls run on the current stream (or `stream`)
of the cache's device and may be captured into a CUDA graph; they record no
gradients. What a call on another stream than the tensors' own was given must
live until that stream has run it.

    k = torch.empty(n_pages, n_kv_heads, page_size, head_dim, dtype=torch.float8_e4m3fn, device="cuda")
    cache = Pages(k, torch.empty_like(k), k_scale, v_scale)   # scales: float32 [n_pages, n_kv_heads, page_size]
    cache.write(table, positions, k_new, v_new)               # [batch, tokens, n_kv_heads, head_dim]
    out = cache.attend(table, lens, q)                        # [batch, tokens, n_q_heads, head_dim]

Position j of sequence b is row j % page_size of page table[b, j // page_size].
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import (DT_BF16, DT_F16, DT_F32, KV_BF16, KV_E4M3, KV_INT8, AttentionStruct, PagesStruct, TableStruct, _check,
               lib)

_FORMAT = {torch.bfloat16: KV_BF16, torch.float8_e4m3fn: KV_E4M3, torch.int8: KV_INT8}
_DTYPE = {torch.float32: DT_F32, torch.bfloat16: DT_BF16, torch.float16: DT_F16}
_byref = ctypes.byref
_ONE = torch.Size((1,))


def _launch(device, stream, call, args):
    """call(stream handle, *args) with `device` current and torch's allocations on that stream."""
    index = device.index
    if stream is None and index == torch.cuda.current_device():
        return call(torch._C._cuda_getCurrentRawStream(index), *args)
    with torch.cuda.device(index):
        if stream is None:
            return call(torch.cuda.current_stream().cuda_stream, *args)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream)) if stream else torch.cuda.default_stream()
        if stream.device.index != index:
            raise ValueError(f"stream of device {stream.device.index}, tensors on device {index}")
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream, *args)


def _copy_call(h, fn, pages, packed, pos, cnt, n, st):
    buf = _CopyBytes.from_buffer_copy(packed)
    at = ctypes.addressof(buf)
    rc = fn(pages, at, pos, cnt, n, at + 24, at + 64, st, h)
    if rc:
        _check(rc)


def _ptr(x, name, shape, dtype, device):
    """data_ptr of a contiguous argument after its checks."""
    if x.dtype is not dtype or x.shape != shape or x.device != device or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got "
                         f"{x.dtype} {tuple(x.shape)} on {x.device}")
    return x.data_ptr()


def _rows(x, name, device):
    """The fields of an mk_rows."""
    dt = _DTYPE.get(x.dtype)
    if dt is None or x.dim() != 4 or x.device != device:
        raise ValueError(f"{name} must be a float32, bfloat16 or float16 tensor [batch, tokens, heads, head_dim] on "
                         f"{device}, got {x.dtype} {tuple(x.shape)} on {x.device}")
    s = x.stride()
    if s[3] != 1 and x.shape[3] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous, got strides {s}")
    return x.data_ptr(), s[0], s[1], s[2], dt, 0


def _written(x, name):
    """Refuses a tensor whose elements share memory by expansion: its rows would be written over one another."""
    s = x.stride()
    if 0 in s and any(n > 1 and not d for n, d in zip(x.shape, s)):
        raise ValueError(f"{name} is written to, but its strides {s} put several elements in one place")


# A call's structures side by side in one buffer: (mk_attention,) mk_page_table, mk_rows, mk_rows
_COPY = struct.Struct("Pqii Pqqqii Pqqqii")
_ATTEND = struct.Struct("PP PPP PP PP ii ff ii Pqii Pqqqii Pqqqii")
_CopyBytes, _AttendBytes = ctypes.c_char * _COPY.size, ctypes.c_char * _ATTEND.size
assert _COPY.size == 24 + 2 * 40 and _ATTEND.size == 96 + _COPY.size and ctypes.sizeof(AttentionStruct) == 96


class Pages:
    """K and V pages: two tensors [n_pages, n_kv_heads, page_size, head_dim] of the same strides (bfloat16,
    float8_e4m3fn or int8, last dimension contiguous) and, for the 8-bit types, two float32 scale tensors
    [n_pages, n_kv_heads, page_size]."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        fmt = _FORMAT.get(k.dtype)
        if fmt is None or v.dtype != k.dtype:
            raise ValueError(f"k and v must both be bfloat16, float8_e4m3fn or int8, got {k.dtype} and {v.dtype}")
        if k.dim() != 4 or v.shape != k.shape or v.stride() != k.stride() or k.stride(3) != 1:
            raise ValueError("k and v must be [n_pages, n_kv_heads, page_size, head_dim] with the same strides and a "
                             "contiguous last dimension")
        if not k.is_cuda or v.device != k.device:
            raise ValueError("k and v must be CUDA tensors of one device")
        if (k_scale is None) != (fmt == KV_BF16) or (v_scale is None) != (fmt == KV_BF16):
            raise ValueError("8-bit pages need k_scale and v_scale, bfloat16 pages have none")
        ss = (0, 0)
        if k_scale is not None:
            for s in (k_scale, v_scale):
                if s.dtype != torch.float32 or s.shape != k.shape[:3] or s.device != k.device or s.stride(2) != 1:
                    raise ValueError("scales must be float32 [n_pages, n_kv_heads, page_size] on the pages' device "
                                     "with a contiguous last dimension")
            if k_scale.stride() != v_scale.stride():
                raise ValueError("k_scale and v_scale must have the same strides")
            ss = k_scale.stride()
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device = k.device
        st = k.stride()
        self._heads = (k.shape[1], k.shape[3])
        self._need = {}  # workspace bytes by shapes
        self._s = PagesStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if k_scale is not None else None,
                              v_scale.data_ptr() if v_scale is not None else None, st[0], st[1], st[2], ss[0], ss[1],
                              fmt, k.shape[0], k.shape[1], k.shape[2], k.shape[3], 0)
        self._at = ctypes.addressof(self._s)

    def _table(self, table):
        s, shape = table.stride(), table.shape
        if table.dtype is not torch.int32 or len(s) != 2 or s[1] != 1 or table.device != self.device:
            raise ValueError(f"table must be an int32 tensor [batch, pages per sequence] on {self.device} with a "
                             f"contiguous last dimension, got {table.dtype} {tuple(table.shape)} on {table.device}")
        return table.data_ptr(), s[0], shape[0], shape[1]

    def _copy(self, fn, table, positions, k, v, counts, status, stream):
        dev, t = self.device, self._table(table)
        rk, rv = _rows(k, "k", dev), _rows(v, "v", dev)
        shape = k.shape
        if shape[0] != t[2] or shape[2:] != self._heads or v.shape != shape:
            raise ValueError(f"k and v must be [{t[2]}, tokens, {self._heads[0]}, {self._heads[1]}], got {tuple(shape)} "
                             f"and {tuple(v.shape)}")
        if positions is None:
            raise ValueError("positions is required")
        pos = _ptr(positions, "positions", shape[:1], torch.int32, dev)
        cnt = 0 if counts is None else _ptr(counts, "counts", shape[:1], torch.int32, dev)
        st = 0 if status is None else _ptr(status, "status", _ONE, torch.int32, dev)
        n = shape[1]
        if shape[0] == 0 or n == 0:
            return
        _launch(dev, stream, _copy_call, (fn, self._at, _COPY.pack(*t, *rk, *rv), pos, cnt, n, st))

    def write(self, table, positions, k, v, counts=None, status=None, stream=None):
        """Rows t < counts[b] (all, without counts) of k and v, [batch, tokens, n_kv_heads, head_dim], to positions
        positions[b] + t, which must be distinct rows of the cache: 8-bit pages get codes and a scale a row.
        positions, counts: int32 [batch]. A position or page out of range is skipped and sets status[0] (int32 [1]) to
        MK_ERR_INVALID_ARG."""
        self._copy(lib().mk_pages_write, table, positions, k, v, counts, status, stream)

    def read(self, table, positions, k, v, counts=None, status=None, stream=None):
        """Fills rows t < counts[b] of k and v, [batch, tokens, n_kv_heads, head_dim], from positions
        positions[b] + t, as code x scale rounded to their type; other rows stay as they are. Returns (k, v)."""
        _written(k, "k")
        _written(v, "v")
        self._copy(lib().mk_pages_read, table, positions, k, v, counts, status, stream)
        return k, v

    def attend(self, table, lens, q, scale=None, softcap=0.0, slopes=None, starts=None, shared_len=0, out=None,
               return_lse=False, status=None, stream=None):
        """Attention of q, [batch, tokens, n_q_heads, head_dim] (bfloat16 or float16): the queries of the last
        `tokens` of the lens[b] cached positions, each over what lies before it and itself.

        lens, starts: int32 [batch] (starts: the first visible position); scale: 1/sqrt(head_dim) by default;
        softcap > 0: scores become softcap * tanh(score / softcap); slopes: float32 [n_q_heads], scores lose
        slope * distance; shared_len: the first positions of all sequences lie in the same pages (whole pages) and
        are read once. A token that sees nothing gets zeros (lse -inf). Returns out, or (out, lse) with lse float32
        [batch, tokens, n_q_heads]. The workspace comes from torch's allocator, on the call's stream."""
        dev, t = self.device, self._table(table)
        rq = _rows(q, "q", dev)
        shape = q.shape
        B, T, Hq, D = shape
        H = self._heads[0]
        if B != t[2] or D != self._heads[1] or Hq < 1 or Hq % H:
            raise ValueError(f"q must be [{t[2]}, tokens, a multiple of {H}, {self._heads[1]}], got {tuple(shape)}")
        if lens is None:
            raise ValueError("lens is required")
        batch = shape[:1]
        n = _ptr(lens, "lens", batch, torch.int32, dev)
        first = 0 if starts is None else _ptr(starts, "starts", batch, torch.int32, dev)
        sl = 0 if slopes is None else _ptr(slopes, "slopes", shape[2:3], torch.float32, dev)
        st = 0 if status is None else _ptr(status, "status", _ONE, torch.int32, dev)
        if out is not None:
            if out.dtype is not q.dtype or out.shape != shape:
                raise ValueError(f"out must have q's type and shape, {q.dtype} {tuple(shape)}")
            _written(out, "out")
        if scale is None:
            scale = 1.0 / math.sqrt(D)
        return _launch(dev, stream, self._attend, (t, rq, q, n, first, sl, st, out, scale, softcap, shared_len,
                                                   return_lse))

    def _attend(self, h, t, rq, q, n, first, sl, st, out, scale, softcap, shared_len, return_lse):
        dev, shape = self.device, q.shape
        B, T, Hq, D = shape
        if out is None:
            out = torch.empty(shape, dtype=q.dtype, device=dev)
            ro = (out.data_ptr(), T * Hq * D, Hq * D, D, rq[4], 0)
        else:
            ro = _rows(out, "out", dev)
        lse = torch.empty(shape[:3], dtype=torch.float32, device=dev) if return_lse else None
        if B and T:
            buf = _AttendBytes()
            at = ctypes.addressof(buf)
            try:
                _ATTEND.pack_into(buf, 0, self._at, at + 96, n, first, sl, at + 120, at + 160,
                                  lse.data_ptr() if return_lse else 0, st, T, Hq, scale, softcap, shared_len, 0, *t, *rq,
                                  *ro)
            except (struct.error, OverflowError) as e:
                raise ValueError(f"scale, softcap and shared_len must be numbers in range: {e}") from None
            L = lib()
            # the workspace's size depends on shapes alone
            key = (B, T, Hq, t[3], shared_len, rq[4])
            need = self._need.get(key)
            if need is None:
                c = ctypes.c_int64()
                _check(L.mk_pages_attend_workspace(at, _byref(c)))
                need = self._need[key] = c.value
            w = torch.empty((need,), dtype=torch.uint8, device=dev) if need else None
            rc = L.mk_pages_attend(at, w.data_ptr() if need else 0, need, h)
            if rc:
                _check(rc)
        return (out, lse) if return_lse else out


class _Memory:
    """Device memory of the library as torch sees it (keeps its owner alive)."""

    def __init__(self, owner, ptr, shape, strides, typestr):
        self.owner = owner
        self.__cuda_array_interface__ = {"shape": shape, "strides": strides, "typestr": typestr, "data": (ptr, False),
                                         "version": 3, "stream": None}


def _device_of(owner, ptr):
    """The device that holds the library's memory at ptr, the current one or another: torch copies what it is asked to
    see on a device that does not hold it, so one byte tells."""
    now = torch.cuda.current_device()
    for i in [now] + [i for i in range(torch.cuda.device_count()) if i != now]:
        if torch.as_tensor(_Memory(owner, ptr, (1,), None, "|u1"), device=f"cuda:{i}").data_ptr() == ptr:
            return torch.device("cuda", i)
    raise RuntimeError(f"no device holds the cache's memory at {ptr:#x}")


def of_cache(kv, layer) -> Pages:
    """The pages of one layer of a model's KVCache (no copy); `.table` is its block table, int32 [batch, pages].
    They hold until the cache is closed."""
    s, t = PagesStruct(), TableStruct()
    _check(lib().mk_kv_view(kv.h, layer, _byref(s), _byref(t)))
    shape = (s.n_pages, s.n_kv_heads, s.page_size, s.head_dim)
    strides = (2 * s.page_stride, 2 * s.head_stride, 2 * s.row_stride, 2)
    # bfloat16 has no type string there: taken as 16-bit integers, then seen as bfloat16
    dev = _device_of(kv, s.k)
    k, v = (torch.as_tensor(_Memory(kv, p, shape, strides, "<i2"), device=dev).view(torch.bfloat16) for p in (s.k, s.v))
    out = Pages(k, v)
    out.table = torch.as_tensor(_Memory(kv, t.table, (t.batch, t.pages_per_seq), None, "<i4"), device=dev)
    return out
