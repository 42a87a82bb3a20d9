"""Latent attention of the caller: rows into a paged latent cache, attention over it, and prompts.

Binding of mk_latent_write, mk_latent_attend and mk_prompt_attend (include/mk.h), for models whose keys and values are
products of one latent vector a token. The absorbed form reads the latents themselves, with queries taken through the
key up-projection and outputs still to be taken through the value up-projection; the expanded form takes keys and
values. As in pages.py everything is the caller's own tensors; calls run on the current stream (or `stream`) of the
tensors' device, may be captured into a CUDA graph, and record no gradients.

    cache = LatentPages(latent, rope)            # [n_pages, page_size, rank] and [n_pages, page_size, rope_dim]
    cache.write(table, positions, rows, gain=norm, inv_freq=freq)       # rows: [batch, tokens, rank + rope_dim]
    out = cache.attend(table, lens, q, q_rope, scale)                   # [batch, tokens, heads, rank]
    out = attend_prompt(q, k, k_rope, v, q_starts, k_starts, scale)     # [tokens, heads, v_dim], a ragged batch

Position j of sequence b is row j % page_size of page table[b, j // page_size].
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import (DT_BF16, DT_F16, LatentAttentionStruct, LatentPagesStruct, PromptAttentionStruct, TableStruct, _check,
               lib)
from .pages import _DTYPE, _ONE, _Memory, _device_of, _launch, _ptr, _rows, _written
from .rotary import _ROTARY, _RotaryBytes, _freq, _layout

_TYPES = {torch.bfloat16: DT_BF16, torch.float16: DT_F16}
_byref = ctypes.byref
_PAGES = struct.Struct("PP qqqq iiiiii")
_WRITE = struct.Struct("Pqii Pqqqii Pii fi")
_ATTEND = struct.Struct("PP PP PPP PP ii fi Pqii Pqqqii Pqqqii Pqqqii 72s")
_PROMPT = struct.Struct("PP PPPPP PP qqqqqqqqq iiiiiiii fi")
_WriteBytes, _AttendBytes = ctypes.c_char * _WRITE.size, ctypes.c_char * _ATTEND.size
_NEED, _KEPT = {}, 256  # workspace bytes by device and shapes, of so many at most
assert _PAGES.size == ctypes.sizeof(LatentPagesStruct) == 72 and _WRITE.size == 24 + 40 + _ROTARY.size
assert _ATTEND.size == 88 + 24 + 3 * 40 + 72 and ctypes.sizeof(LatentAttentionStruct) == 88
assert _PROMPT.size == ctypes.sizeof(PromptAttentionStruct) == 184


class LatentPages:
    """A layer's latent cache: latent [n_pages, page_size, rank] and rope [n_pages, page_size, rope_dim], both bfloat16
    or both float16, last dimensions contiguous (the two may be parts of one tensor)."""

    def __init__(self, latent, rope):
        dtype, shape, rs = latent.dtype, latent.shape, rope.shape
        dt = _TYPES.get(dtype)
        if dt is None or rope.dtype is not dtype:
            raise ValueError(f"latent and rope must both be bfloat16 or float16, got {latent.dtype} and {rope.dtype}")
        ls, ss = latent.stride(), rope.stride()
        if len(shape) != 3 or len(rs) != 3 or rs[:2] != shape[:2] or ls[2] != 1 or ss[2] != 1:
            raise ValueError("latent must be [n_pages, page_size, rank], rope [n_pages, page_size, rope_dim], with "
                             "contiguous last dimensions")
        self.device = latent.device
        if not latent.is_cuda or rope.device != self.device:
            raise ValueError("latent and rope must be CUDA tensors of one device")
        self.latent, self.rope = latent, rope
        n, ps, self.rank = shape
        self.rope_dim = rs[2]
        # the mk_latent_pages of the calls
        self._s = _PAGES.pack(latent.data_ptr(), rope.data_ptr(), ls[0], ls[1], ss[0], ss[1], dt, n, ps, self.rank,
                              self.rope_dim, 0)
        self._key = (self.device.index, ps, self.rank, dt, min(ls[0], ls[1], ss[0], ss[1]) > 0)

    def _table(self, table):
        s, shape = table.stride(), table.shape
        if table.dtype is not torch.int32 or len(s) != 2 or s[1] != 1 or table.device != self.device:
            raise ValueError(f"table must be an int32 tensor [batch, pages per sequence] on {self.device} with a "
                             f"contiguous last dimension, got {table.dtype} {tuple(table.shape)} on {table.device}")
        return table.data_ptr(), s[0], shape[0], shape[1]

    def write(self, table, positions, rows, gain=None, eps=1e-6, inv_freq=None, layout="half", magnitude=1.0,
              counts=None, status=None, stream=None):
        """Rows t < counts[b] (all, without counts) of `rows`, [batch, tokens, rank + rope_dim] (float32, bfloat16 or
        float16), to positions positions[b] + t, which must be distinct rows of the cache.

        gain: [rank] of any of these types, the latent part becomes x / sqrt(mean x^2 + eps) * gain; without it, it is
        kept. inv_freq: float64 [rope_dim / 2], the rope part turns by its position as in rotary.rotate; without it,
        it is kept. positions, counts: int32 [batch]. A position or page out of range is skipped and sets status[0]
        (int32 [1]) to MK_ERR_INVALID_ARG."""
        dev, t = self.device, self._table(table)
        dt = _DTYPE.get(rows.dtype)
        if dt is None or rows.dim() != 3 or rows.device != dev or (rows.shape[2] > 1 and rows.stride(2) != 1):
            raise ValueError(f"rows must be a float32, bfloat16 or float16 tensor [batch, tokens, rank + rope_dim] on "
                             f"{dev} with a contiguous last dimension, got {rows.dtype} {tuple(rows.shape)} on {rows.device}")
        shape, s = rows.shape, rows.stride()
        if shape[0] != t[2] or shape[2] != self.rank + self.rope_dim:
            raise ValueError(f"rows must be [{t[2]}, tokens, {self.rank + self.rope_dim}], got {tuple(shape)}")
        if positions is None:
            raise ValueError("positions is required")
        pos = _ptr(positions, "positions", shape[:1], torch.int32, dev)
        cnt = 0 if counts is None else _ptr(counts, "counts", shape[:1], torch.int32, dev)
        st = 0 if status is None else _ptr(status, "status", _ONE, torch.int32, dev)
        g = gdt = 0
        if gain is not None:
            gdt = _DTYPE.get(gain.dtype)
            if gdt is None or gain.shape != (self.rank,) or gain.device != dev or not gain.is_contiguous():
                raise ValueError(f"gain must be a contiguous float32, bfloat16 or float16 tensor ({self.rank},) on {dev}")
            g = gain.data_ptr()
        f, n, code = 0, 0, 0
        if inv_freq is not None:
            f, n = _freq(inv_freq, dev)
            code = _layout(layout)
        if shape[0] == 0 or shape[1] == 0:
            return
        try:
            packed = _WRITE.pack(*t, rows.data_ptr(), s[0], s[1], 0, dt, 0, f, n, code, magnitude, 0)
            eps = float(eps)
        except (struct.error, OverflowError, TypeError) as e:
            raise ValueError(f"eps and magnitude must be numbers in range: {e}") from None
        _launch(dev, stream, self._write, (packed, pos, cnt, shape[1], g, gdt, eps, f != 0, st))

    def _write(self, h, packed, pos, cnt, n, g, gdt, eps, turned, st):
        buf = _WriteBytes.from_buffer_copy(packed)
        at = ctypes.addressof(buf)
        rc = lib().mk_latent_write(self._s, at, pos, cnt, n, at + 24, g, gdt, eps, at + 64 if turned else 0, st, h)
        if rc:
            _check(rc)

    def attend(self, table, lens, q, q_rope, scale, starts=None, out=None, return_lse=False, status=None, stream=None):
        """Attention, in the latent space, of the queries of the last `tokens` of the lens[b] cached positions, each
        over what lies before it and itself: q [batch, tokens, heads, rank] against the latents and q_rope [batch,
        tokens, heads, rope_dim] against the rope parts, of the cache's type.

        lens, starts: int32 [batch] (starts: the first visible position); scale: of the summed products, such as
        1/sqrt of the unabsorbed head's size. A token that sees nothing gets zeros (lse -inf). Returns out, shaped as
        q, or (out, lse) with lse float32 [batch, tokens, heads]. The workspace comes from torch's allocator, on the
        call's stream."""
        dev, t = self.device, self._table(table)
        rq, rr = _rows(q, "q", dev), _rows(q_rope, "q_rope", dev)
        shape = q.shape
        if shape[0] != t[2] or shape[3] != self.rank or q_rope.shape != shape[:3] + (self.rope_dim,):
            raise ValueError(f"q must be [{t[2]}, tokens, heads, {self.rank}], q_rope the same with {self.rope_dim} "
                             f"values, got {tuple(shape)} and {tuple(q_rope.shape)}")
        if q.dtype is not self.latent.dtype or q_rope.dtype is not q.dtype:
            raise ValueError(f"q and q_rope must have the cache's type, {self.latent.dtype}")
        if lens is None:
            raise ValueError("lens is required")
        batch = shape[:1]
        n = _ptr(lens, "lens", batch, torch.int32, dev)
        first = 0 if starts is None else _ptr(starts, "starts", batch, torch.int32, dev)
        st = 0 if status is None else _ptr(status, "status", _ONE, torch.int32, dev)
        if out is not None:
            if out.dtype is not q.dtype or out.shape != shape:
                raise ValueError(f"out must have q's type and shape, {q.dtype} {tuple(shape)}")
            _written(out, "out")
        return _launch(dev, stream, self._attend, (t, rq, rr, q, n, first, st, out, scale, return_lse))

    def _attend(self, h, t, rq, rr, q, n, first, st, out, scale, return_lse):
        dev, shape = self.device, q.shape
        B, T, H, R = shape
        if out is None:
            out = torch.empty(shape, dtype=q.dtype, device=dev)
            ro = (out.data_ptr(), T * H * R, H * R, R, rq[4], 0)
        else:
            ro = _rows(out, "out", dev)
        lse = torch.empty(shape[:3], dtype=torch.float32, device=dev) if return_lse else None
        if B and T and H:
            buf = _AttendBytes()
            at = ctypes.addressof(buf)
            try:
                _ATTEND.pack_into(buf, 0, at + 232, at + 88, n, first, at + 112, at + 152, at + 192,
                                  lse.data_ptr() if return_lse else 0, st, T, H, scale, 0, *t, *rq, *rr, *ro, self._s)
            except (struct.error, OverflowError) as e:
                raise ValueError(f"scale must be a number in range: {e}") from None
            L = lib()
            key = (self._key, B, T, H, t[3])  # the workspace's size depends on shapes alone
            need = _NEED.get(key)
            if need is None:
                c = ctypes.c_int64()
                _check(L.mk_latent_attend_workspace(at, _byref(c)))
                if len(_NEED) >= _KEPT:
                    _NEED.clear()
                need = _NEED[key] = c.value
            w = torch.empty((need,), dtype=torch.uint8, device=dev) if need else None
            rc = L.mk_latent_attend(at, w.data_ptr() if need else 0, need, h)
            if rc:
                _check(rc)
        return (out, lse) if return_lse else out


def of_cache(kv, layer) -> LatentPages:
    """The latent cache of one layer of a model's KVCache (no copy); `.table` is its block table, int32 [batch, pages].
    They hold until the cache is closed."""
    s, t = LatentPagesStruct(), TableStruct()
    _check(lib().mk_kv_latent_view(kv.h, layer, _byref(s), _byref(t)))
    dev = _device_of(kv, s.latent)

    def part(ptr, width, page, row):
        # bfloat16 has no type string there: taken as 16-bit integers, then seen as bfloat16
        m = _Memory(kv, ptr, (s.n_pages, s.page_size, width), (2 * page, 2 * row, 2), "<i2")
        return torch.as_tensor(m, device=dev).view(torch.bfloat16)

    out = LatentPages(part(s.latent, s.rank, s.page_stride, s.row_stride),
                      part(s.rope, s.rope_dim, s.rope_page_stride, s.rope_row_stride))
    out.table = torch.as_tensor(_Memory(kv, t.table, (t.batch, t.pages_per_seq), None, "<i4"), device=dev)
    return out


def _wide(x, name, dims, dtype, device):
    """data_ptr and strides of a tensor of `dims` dimensions with a contiguous last one."""
    if x.dim() != dims or x.dtype is not dtype or x.device != device or (x.stride(-1) != 1 and x.shape[-1] > 1):
        raise ValueError(f"{name} must be a {dtype} tensor of {dims} dimensions on {device} with a contiguous last one, "
                         f"got {x.dtype} {tuple(x.shape)} on {x.device}")
    return x.data_ptr(), x.stride()


def attend_prompt(q, k, k_rope, v, q_starts, k_starts, scale, out=None, return_lse=False, status=None, stream=None):
    """Causal attention of a ragged batch over expanded keys and values: q [tokens, heads, nope + rope], k [keys, heads,
    nope], k_rope [keys, rope] (shared by the heads), v [keys, heads, v_dim], all bfloat16 or all float16.

    q_starts, k_starts: int32 [batch + 1], ascending: sequence b has rows q_starts[b] .. q_starts[b+1] - 1 of q and out
    and rows k_starts[b] .. k_starts[b+1] - 1 of the keys. Its queries are the last of its positions: query i of n over
    m keys sees keys 0 .. m - n + i. A query that sees nothing gets zeros (lse -inf). Returns out [tokens, heads,
    v_dim], or (out, lse) with lse float32 [tokens, heads]; rows of no sequence are left as they were (in a new tensor:
    undefined). Bounds that descend or leave the rows skip the sequence and set status[0] (int32 [1]) to
    MK_ERR_INVALID_ARG. Supported: nope 128, rope 64, v_dim 128."""
    dt = _TYPES.get(q.dtype)
    if dt is None or q.dim() != 3 or not q.is_cuda:
        raise ValueError(f"q must be a bfloat16 or float16 CUDA tensor [tokens, heads, nope + rope], got {q.dtype} "
                         f"{tuple(q.shape)} on {q.device}")
    dev, dtype = q.device, q.dtype
    (pq, sq), (pk, sk) = _wide(q, "q", 3, dtype, dev), _wide(k, "k", 3, dtype, dev)
    (pr, sr), (pv, sv) = _wide(k_rope, "k_rope", 2, dtype, dev), _wide(v, "v", 3, dtype, dev)
    N, H, D = q.shape
    M, _, nope = k.shape
    rope, vd = k_rope.shape[1], v.shape[2]
    if k.shape[1] != H or v.shape[:2] != k.shape[:2] or k_rope.shape[0] != M or D != nope + rope:
        raise ValueError(f"k must be [keys, {H}, nope], k_rope [keys, rope], v [keys, {H}, v_dim] with nope + rope = {D}, "
                         f"got {tuple(k.shape)}, {tuple(k_rope.shape)} and {tuple(v.shape)}")
    if q_starts is None or k_starts is None or q_starts.dim() != 1 or q_starts.shape[0] < 2:
        raise ValueError("q_starts and k_starts must be [batch + 1], batch at least 1")
    qs = _ptr(q_starts, "q_starts", q_starts.shape, torch.int32, dev)
    ks = _ptr(k_starts, "k_starts", q_starts.shape, torch.int32, dev)
    st = 0 if status is None else _ptr(status, "status", _ONE, torch.int32, dev)
    if out is not None:
        if out.shape != (N, H, vd):
            raise ValueError(f"out must be [{N}, {H}, {vd}], got {tuple(out.shape)}")
        _wide(out, "out", 3, dtype, dev)
        _written(out, "out")
    return _launch(dev, stream, _prompt, (pq, sq, pk, sk, pr, sr, pv, sv, qs, ks, st, dt, (N, M, H, nope, rope, vd),
                                          q_starts.shape[0] - 1, scale, out, return_lse, dtype, dev))


def _prompt(h, pq, sq, pk, sk, pr, sr, pv, sv, qs, ks, st, dt, dims, batch, scale, out, return_lse, dtype, dev):
    N, M, H, nope, rope, vd = dims
    if out is None:
        out = torch.empty((N, H, vd), dtype=dtype, device=dev)
    lse = torch.empty((N, H), dtype=torch.float32, device=dev) if return_lse else None
    if N and H:
        so = out.stride()
        try:
            a = _PROMPT.pack(qs, ks, pq, pk, pr, pv, out.data_ptr(), lse.data_ptr() if return_lse else 0, st, sq[0],
                             sq[1], sk[0], sk[1], sr[0], sv[0], sv[1], so[0], so[1], batch, N, M, H, nope, rope, vd, dt,
                             scale, 0)
        except (struct.error, OverflowError) as e:
            raise ValueError(f"scale must be a number in range: {e}") from None
        rc = lib().mk_prompt_attend(a, h)
        if rc:
            _check(rc)
    return (out, lse) if return_lse else out
