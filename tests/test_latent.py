"""Latent caches of the caller: rows in, attention over them, against the definitions in 64 bits.

Tolerances. Writing: a sum of up to 1024 squares in 32 bits, its root and three products lose less than 2^-18 of a latent
value; the rope part turns as in test_rotary; each is rounded once to the cache's type (eps/2; fp16: at least 2^-25).
Attention: a score is a sum of rank + 64 products, exact in 32 bits each, whose sum and scaling lose at most
(rank + 72) 2^-23 of sum |q k| scale; e^x turns that into a relative error of every weight, softmax normalises (a
factor 2). A weight goes in rounded to the cache's type: eps/2 of it, in fp16 at least 2^-25 of the largest. 32-bit sums
and the join of pieces add less than 2^-18, and the result is rounded to its type.
"""
import ctypes
import math

import pytest
import torch

import moe_decode_megakernel_02_gb300 as mk
from moe_decode_megakernel_02_gb300 import latent, rotary
from test_rotary import expected as turned

gpu = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


def make_cache(dtype, n, ps, rank=512, rope=64, seed=0, together=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if together:  # parts of one row
        x = torch.randn((n, ps, rank + rope), generator=g, device="cuda").to(dtype)
        return latent.LatentPages(x[..., :rank], x[..., rank:])
    return latent.LatentPages(*(torch.randn((n, ps, w), generator=g, device="cuda").to(dtype) for w in (rank, rope)))


def make_table(B, cols, n, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(n, generator=g)[:B * cols].to(torch.int32).view(B, cols).cuda()


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def queries(dtype, B, T, H, rank=512, rope=64, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return tuple(torch.randn((B, T, H, w), generator=g, device="cuda").to(dtype) for w in (rank, rope))


def check_attend(cache, table, lens, q, qr, scale, starts=None, given=None, **kw):
    """A call (or what one gave) against the definition."""
    out, lse = given or cache.attend(table, lens, q, qr, scale, starts=starts, return_lse=True, **kw)
    B, T, H, R = q.shape
    ps = cache.latent.shape[1]
    dtype = q.dtype
    half = torch.finfo(dtype).eps / 2
    for b in range(B):
        n = min(lens[b].item(), table.shape[1] * ps)
        pg = table[b, :-(-n // ps)].long() if n > 0 else table[b, :0].long()
        c, r = (x[pg].reshape(-1, x.shape[2])[:max(n, 0)].double() for x in (cache.latent, cache.rope))
        first = 0 if starts is None else max(starts[b].item(), 0)
        for t in range(T):
            end = min(lens[b].item() - T + t + 1, n)
            if end <= first:
                assert (out[b, t] == 0).all() and (lse[b, t] == -math.inf).all()
                continue
            cc, rr, qq, qq2 = c[first:end], r[first:end], q[b, t].double(), qr[b, t].double()
            x = (qq @ cc.T + qq2 @ rr.T) * scale
            size = (qq.abs() @ cc.abs().T + qq2.abs() @ rr.abs().T).amax(-1) * abs(scale)
            e = (R + 72) * 2.0 ** -23 * size
            w = torch.softmax(x, -1)
            want = w @ cc
            bound = (w @ cc.abs()) * (2 * e + half + 2.0 ** -18)[:, None]
            if dtype == torch.float16:
                bound += 2.0 ** -25 * (cc.abs().sum(0) + 1)
            bound += want.abs() * half
            err = (out[b, t].double() - want).abs()
            assert (err <= bound).all(), (b, t, (err / bound).max().item())
            want = torch.logsumexp(x, -1)
            assert ((lse[b, t].double() - want).abs() <= e + 2.0 ** -18 + want.abs() * 2.0 ** -22).all()
    return out, lse


# ---------------------------------------------------------------- refusals (CPU)

def _structs(**over):
    one = 4096  # an address that is aligned and never followed
    p = dict(latent=one, rope=one, page_stride=64 * 512, row_stride=512, rope_page_stride=64 * 64, rope_row_stride=64,
             dtype=mk.DT_BF16, n_pages=8, page_size=64, rank=512, rope_dim=64, reserved=0)
    t = dict(table=one, stride=4, batch=2, pages_per_seq=4)
    q, r, o = (dict(data=one, seq_stride=8192, token_stride=8192, head_stride=512, dtype=mk.DT_BF16, reserved=0)
               for _ in range(3))
    a = dict(lens=one, starts=None, lse=None, status=None, n_tokens=1, n_heads=16, scale=0.125, reserved=0)
    y = dict(inv_freq=one, n=64, layout=mk.ROTARY_HALF, magnitude=1.0, inverse=0)
    groups = {"p": p, "t": t, "q": q, "r": r, "o": o, "a": a, "y": y}
    for key, val in over.items():
        group, name = key.split("__")
        groups[group][name] = val
    return (mk.LatentPagesStruct(**p), mk.TableStruct(**t), mk.RowsStruct(**q), mk.RowsStruct(**r), mk.RowsStruct(**o), a,
            mk.RotaryStruct(**y))


BAD_PAGES = [
    (dict(p__latent=None), mk.ERR_INVALID_ARG), (dict(p__rope=None), mk.ERR_INVALID_ARG),
    (dict(p__dtype=mk.DT_F32), mk.ERR_INVALID_ARG), (dict(p__latent=4104), mk.ERR_INVALID_ARG),
    (dict(p__rope=4104), mk.ERR_INVALID_ARG), (dict(p__row_stride=516), mk.ERR_INVALID_ARG),
    (dict(p__rope_row_stride=68), mk.ERR_INVALID_ARG), (dict(p__page_stride=-64), mk.ERR_INVALID_ARG),
    (dict(p__n_pages=0), mk.ERR_INVALID_ARG), (dict(p__rank=0), mk.ERR_INVALID_ARG),
    (dict(p__rank=500), mk.ERR_UNSUPPORTED), (dict(p__rank=1032), mk.ERR_UNSUPPORTED),
    (dict(p__rope_dim=264), mk.ERR_UNSUPPORTED), (dict(p__rope_dim=0), mk.ERR_INVALID_ARG),
    (dict(p__page_size=48), mk.ERR_UNSUPPORTED), (dict(p__page_size=0), mk.ERR_UNSUPPORTED),
    (dict(t__table=None), mk.ERR_INVALID_ARG), (dict(t__table=4098), mk.ERR_INVALID_ARG),
    (dict(t__batch=0), mk.ERR_INVALID_ARG), (dict(t__pages_per_seq=0), mk.ERR_INVALID_ARG),
    (dict(t__stride=-1), mk.ERR_INVALID_ARG), (dict(t__pages_per_seq=1 << 25), mk.ERR_UNSUPPORTED),
    (dict(t__batch=1 << 21), mk.ERR_UNSUPPORTED),
]


def _attention(p, t, q, r, o, a):
    ptr = ctypes.pointer
    return mk.LatentAttentionStruct(pages=ptr(p), table=ptr(t), q=ptr(q), q_rope=ptr(r), out=ptr(o), **a)


@pytest.mark.parametrize("over,code", BAD_PAGES)
def test_bad_pages_are_refused(over, code):
    p, t, q, r, o, a, y = _structs(**over)
    ref, L = ctypes.byref, mk.lib()
    assert L.mk_latent_write(ref(p), ref(t), 4096, None, 1, ref(q), None, 0, 1e-6, None, None, None) == code
    assert L.mk_last_error()
    att = _attention(p, t, q, r, o, a)
    assert L.mk_latent_attend(ref(att), 4096, 1 << 40, None) == code


@pytest.mark.parametrize("over,code", [
    (dict(a__n_tokens=0), mk.ERR_INVALID_ARG), (dict(a__n_heads=0), mk.ERR_INVALID_ARG),
    (dict(a__lens=None), mk.ERR_INVALID_ARG), (dict(a__lens=4098), mk.ERR_INVALID_ARG),
    (dict(a__lse=4098), mk.ERR_INVALID_ARG), (dict(a__scale=math.nan), mk.ERR_INVALID_ARG),
    (dict(a__scale=math.inf), mk.ERR_INVALID_ARG),
    (dict(q__data=None), mk.ERR_INVALID_ARG), (dict(r__data=None), mk.ERR_INVALID_ARG),
    (dict(o__data=None), mk.ERR_INVALID_ARG), (dict(q__data=4097), mk.ERR_INVALID_ARG),
    (dict(q__dtype=mk.DT_F16), mk.ERR_INVALID_ARG), (dict(r__dtype=mk.DT_F32), mk.ERR_INVALID_ARG),
    (dict(o__dtype=mk.DT_F16), mk.ERR_INVALID_ARG), (dict(p__rank=128), mk.ERR_UNSUPPORTED),
    (dict(p__rope_dim=32), mk.ERR_UNSUPPORTED), (dict(a__n_heads=1 << 30), mk.ERR_UNSUPPORTED),
])
def test_bad_attention_arguments_are_refused(over, code):
    p, t, q, r, o, a, y = _structs(**over)
    att, n = _attention(p, t, q, r, o, a), ctypes.c_int64()
    assert mk.lib().mk_latent_attend(ctypes.byref(att), 4096, 1 << 40, None) == code
    assert mk.lib().mk_latent_attend_workspace(ctypes.byref(att), ctypes.byref(n)) == code


def test_bad_writes_are_refused():
    p, t, q, r, o, a, y = _structs()
    ref, L, bad = ctypes.byref, mk.lib(), mk.ERR_INVALID_ARG

    def write(pages=p, table=t, positions=4096, counts=None, n=1, rows=q, gain=None, gdt=mk.DT_BF16, eps=1e-6, rot=None,
              status=None):
        return L.mk_latent_write(pages and ref(pages), table and ref(table), positions, counts, n, rows and ref(rows),
                                 gain, gdt, eps, rot and ref(rot), status, None)

    assert write(pages=None) == bad and write(table=None) == bad and write(positions=None) == bad
    assert write(positions=4098) == bad and write(counts=4098) == bad and write(status=4098) == bad
    assert write(n=-1) == bad and write(rows=None) == bad and write(gain=4097) == bad and write(gain=4096, gdt=7) == bad
    assert write(gain=4096, eps=-1.0) == bad and write(gain=4096, eps=math.nan) == bad
    for over in (dict(y__n=32), dict(y__n=63), dict(y__inv_freq=None), dict(y__layout=2), dict(y__magnitude=math.nan)):
        assert write(rot=_structs(**over)[6]) == bad
    assert write(n=0) == mk.OK
    assert L.mk_latent_attend(None, 4096, 1 << 40, None) == bad
    assert L.mk_latent_attend_workspace(None, None) == bad
    assert L.mk_kv_latent_view(None, 0, ref(p), ref(t)) == bad


# ---------------------------------------------------------------- writing

@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,T,ps,rank,rope,layout,normed", [
    (1, 1, 64, 512, 64, "half", True), (3, 7, 16, 512, 64, "interleaved", True), (5, 40, 8, 256, 32, "half", False),
    (2, 3, 1, 128, 16, "interleaved", True), (2, 33, 128, 1024, 256, "half", True), (4, 9, 32, 72, 8, "half", True),
    (2, 600, 64, 512, 64, "half", True),
])
def test_write(dtype, rows, B, T, ps, rank, rope, layout, normed):
    g = torch.Generator(device="cuda").manual_seed(B * T)
    cols = -(-(T + 2 * ps + 3) // ps)
    cache = make_cache(dtype, B * cols + 2, ps, rank, rope)
    before = cache.latent.clone(), cache.rope.clone()
    table = make_table(B, cols, B * cols + 2)
    x = (torch.randn((B, T, rank + rope), generator=g, device="cuda") * 3).to(rows)
    gain = (1 + 0.2 * torch.randn((rank,), generator=g, device="cuda")).to(dtype) if normed else None
    pos = torch.randint(0, 2 * ps + 3, (B,), generator=g, device="cuda").to(torch.int32)
    counts = torch.randint(0, T + 1, (B,), generator=g, device="cuda").to(torch.int32)
    counts[0] = T
    freq = rotary.frequencies(rope)
    status = ints(0)
    cache.write(table, pos, x, gain=gain, eps=1e-5, inv_freq=freq, layout=layout, counts=counts, status=status)
    assert status.item() == 0
    want_c, want_r = before[0].double(), before[1].double()
    size_r = torch.zeros_like(want_r)
    half = torch.finfo(dtype).eps / 2
    seen = torch.zeros(want_c.shape[:2], dtype=torch.bool, device="cuda")
    for b in range(B):
        n = counts[b].item()
        at = pos[b] + torch.arange(n, device="cuda")
        page, row = table[b, at // ps].long(), at % ps
        c = x[b, :n, :rank].double()
        if normed:
            c = c / (c.square().mean(-1, keepdim=True) + 1e-5).sqrt() * gain.double()
        want_c[page, row] = c
        v, s = turned(x[None, b, :n, None, rank:], at[None], freq, layout, 0)
        want_r[page, row], size_r[page, row] = v[0, :, 0], s[0, :, 0]
        seen[page, row] = True
    least = 2.0 ** -25 if dtype == torch.float16 else 0.0
    err = (cache.latent.double() - want_c).abs()
    assert (err <= want_c.abs() * (half + (2.0 ** -18 if normed else 0)) + least).all()
    assert ((cache.rope.double() - want_r).abs() <= size_r * 2.0 ** -21 + want_r.abs() * (half + 2.0 ** -21) + least).all()
    # every other row is as it was
    assert torch.equal(cache.latent[~seen], before[0][~seen]) and torch.equal(cache.rope[~seen], before[1][~seen])


@gpu
def test_write_of_parts_of_wider_rows_and_kept_rope():
    """Unaligned rows of a fused projection, a gain of another type, no rotation: values as they are."""
    cache = make_cache(torch.bfloat16, 9, 16, together=True)
    table = make_table(2, 4, 9)
    x = torch.randn((2, 5, 700), device="cuda").bfloat16()[..., 3:579]
    gain = torch.rand((512,), device="cuda")
    cache.write(table, ints(0, 30), x, gain=gain)
    for b, first in ((0, 0), (1, 30)):
        at = first + torch.arange(5, device="cuda")
        page, row = table[b, at // 16].long(), at % 16
        c = x[b, :, :512].double()
        want = c / (c.square().mean(-1, keepdim=True) + 1e-6).sqrt() * gain.double()
        assert ((cache.latent[page, row].double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -18)).all()
        assert torch.equal(cache.rope[page, row], x[b, :, 512:])


@gpu
def test_write_skips_what_is_out_of_range():
    cache = make_cache(torch.bfloat16, 6, 16)
    before = cache.latent.clone(), cache.rope.clone()
    table = ints(0, 99, 1, -1).view(2, 2)  # second pages do not exist
    x = torch.randn((2, 20, 576), device="cuda").bfloat16()
    status = ints(0)
    cache.write(table, ints(10, -4), x, status=status)
    assert status.item() == mk.ERR_INVALID_ARG
    assert torch.equal(cache.latent[0, 10:], x[0, :6, :512]) and torch.equal(cache.rope[1, :16], x[1, 4:20, 512:])
    cache.latent[0, 10:], cache.latent[1], cache.rope[0, 10:], cache.rope[1] = before[0][0, 10:], before[0][1], before[1][0, 10:], before[1][1]
    assert torch.equal(cache.latent, before[0]) and torch.equal(cache.rope, before[1])


# ---------------------------------------------------------------- attention

@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,T,H,L,ps", [
    (1, 1, 16, 1, 64), (1, 1, 16, 63, 64), (1, 1, 16, 64, 64), (1, 1, 1, 65, 16), (2, 1, 16, 129, 16), (3, 2, 5, 300, 32),
    (1, 1, 16, 5000, 64), (8, 7, 16, 700, 64), (2, 1, 128, 400, 64), (2, 3, 40, 257, 128), (1, 33, 8, 500, 64),
    (40, 1, 16, 333, 64), (1, 5, 13, 1111, 8), (2, 2, 9, 100, 1), (1, 4, 16, 900, 1024), (1, 1, 200, 130, 64),
])
def test_attend(dtype, B, T, H, L, ps):
    g = torch.Generator().manual_seed(L)
    cols = -(-L // ps)
    cache = make_cache(dtype, B * cols + 1, ps)
    table = make_table(B, cols, B * cols + 1)
    lens = torch.randint(1, L + 1, (B,), generator=g).to(torch.int32).cuda()
    lens[0] = L
    q, qr = queries(dtype, B, T, H)
    check_attend(cache, table, lens, q, qr, 192 ** -0.5)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,ps", [(1, 16, 64), (7, 16, 64), (3, 5, 16)])
def test_attend_rank_256(dtype, T, H, ps):
    cache = make_cache(dtype, 64, ps, rank=256)
    table = make_table(3, 20, 64)
    q, qr = queries(dtype, 3, T, H, rank=256)
    check_attend(cache, table, ints(20 * ps, 5 * ps + 3, 2), q, qr, 0.07)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_attend_masks(dtype):
    """Late starts, paddings, tokens before the first position, starts past the end, lengths beyond the table."""
    cache = make_cache(dtype, 80, 16)
    table = make_table(8, 9, 80)
    q, qr = queries(dtype, 8, 3, 6)
    lens = ints(100, 0, 2, 144, 60, 1, -5, 70)
    starts = ints(33, 0, 0, 143, 60, -7, 3, 69)
    check_attend(cache, table, lens, q, qr, 0.05, starts=starts)
    # every sequence empty: one launch all the same
    out, lse = cache.attend(table, torch.zeros_like(lens), q, qr, 0.05, return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    status = ints(0)
    check_attend(cache, table, ints(100, 0, 2, 500, 60, 1, -5, 70), q, qr, 0.05, status=status)
    assert status.item() == mk.ERR_INVALID_ARG


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf, 65504.0])
def test_what_a_row_does_not_see_cannot_reach_it(dtype, junk):
    """Everything but the rows that are seen holds junk: pages of nobody, rows behind the length, before the start."""
    ps, L, T, H = 16, 100, 2, 16
    cache = make_cache(dtype, 30, ps)
    table = make_table(3, 8, 30)
    lens, starts = ints(L, 37, 64), ints(0, 21, 63)
    q, qr = queries(dtype, 3, T, H)
    seen = torch.zeros(cache.latent.shape[:2], dtype=torch.bool, device="cuda")
    for b in range(3):
        at = torch.arange(starts[b].item(), lens[b].item(), device="cuda")
        seen[table[b, at // ps].long(), at % ps] = True
    cache.latent[~seen] = junk
    cache.rope[~seen] = junk
    check_attend(cache, table, lens, q, qr, 0.06, starts=starts)
    # the newest position alone: token 0 of each sequence must not take it
    last = lens - 1
    for b in range(3):
        cache.latent[table[b, last[b] // ps].long(), last[b] % ps] = junk
    got = cache.attend(table, lens, q, qr, 0.06, starts=starts)
    clean = latent.LatentPages(torch.where(seen[..., None], cache.latent, 0).nan_to_num(0, 0, 0), cache.rope.nan_to_num(0, 0, 0))
    want = clean.attend(table, lens, q, qr, 0.06, starts=starts)
    assert torch.equal(got[:, 0], want[:, 0])


@gpu
def test_attend_pages_that_do_not_exist_count_as_zeros():
    cache = make_cache(torch.bfloat16, 10, 16)
    table = make_table(2, 4, 10)
    bad = table.clone()
    bad[0, 1], bad[1, 3] = 10, -1
    q, qr = queries(torch.bfloat16, 2, 2, 16)
    lens, status = ints(60, 64), ints(0)
    out = cache.attend(bad, lens, q, qr, 0.06, status=status)
    assert status.item() == mk.ERR_INVALID_ARG
    wide = latent.LatentPages(torch.cat([cache.latent, 0 * cache.latent[:1]]), torch.cat([cache.rope, 0 * cache.rope[:1]]))
    bad[0, 1] = bad[1, 3] = 10
    assert torch.equal(out, wide.attend(bad, lens, q, qr, 0.06))


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_attend_scores_far_apart_and_equal(dtype):
    """One position takes all; weights rise by 2^8 and more from tile to tile; all weights equal; a negative scale."""
    cache = make_cache(dtype, 33, 64)
    table = make_table(1, 32, 33)
    lens = ints(2000)
    q, qr = queries(dtype, 1, 1, 16)
    for scale in (3.0, -0.3, 0.0):
        check_attend(cache, table, lens, q, qr, scale)
    j = torch.arange(2048, device="cuda", dtype=torch.float32)
    for slope in (0.2, -0.2):  # growing or falling scores
        cache.rope[table[0].long()] = 0
        cache.rope[table[0].long(), :, 0] = (j * slope).view(32, 64).to(dtype)
        qr[..., 0] = 1
        check_attend(cache, table, lens, 0 * q, qr, 1.0)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offset", [0, 1])
def test_attend_strides(dtype, offset):
    """Cache parts of one tensor with its pages apart, queries of heads before tokens, an output inside a wider one."""
    ps, n = 32, 20
    pool = torch.randn((n, 2, ps, 584), device="cuda").to(dtype)
    cache = latent.LatentPages(pool[:, 1, :, 8:520], pool[:, 0, :, 520:584])
    table = make_table(2, 9, n)
    wide = torch.randn((2, 6, 3, 700), device="cuda").to(dtype).transpose(1, 2)  # [2, 3, 6, 700]
    q, qr = wide[..., offset:512 + offset], wide[..., 600 + offset:664 + offset]
    lens = ints(288, 100)
    want, _ = check_attend(cache, table, lens, q, qr, 0.06)
    room = torch.full((2, 6, 3, 514), 7.0, device="cuda").to(dtype).transpose(1, 2)
    out = room[..., offset:512 + offset]
    assert cache.attend(table, lens, q, qr, 0.06, out=out) is out
    assert torch.equal(out, want)
    out[:] = 7.0
    assert (room == 7.0).all()


@gpu
def test_attend_far_pages():
    """Offsets past 2^31 elements and 2^32 bytes."""
    n, ps = 4300, 1024
    pool = torch.empty((n, ps, 576), dtype=torch.bfloat16, device="cuda")  # 5 GB
    cache = latent.LatentPages(pool[..., :512], pool[..., 512:])
    table = ints(n - 1, 0, n - 2).view(1, 3)
    x = torch.randn((1, 3 * ps, 576), device="cuda").bfloat16()
    cache.write(table, ints(0), x)
    assert torch.equal(pool[n - 1], x[0, :ps]) and torch.equal(pool[n - 2], x[0, 2 * ps:])
    q, qr = queries(torch.bfloat16, 1, 1, 16)
    check_attend(cache, table, ints(2900), q, qr, 0.06)


@gpu
def test_attend_captured_on_streams_and_side_by_side():
    cache = make_cache(torch.bfloat16, 400, 64)
    table = make_table(4, 90, 400)
    q, qr = queries(torch.bfloat16, 4, 2, 16)
    lens = ints(5000, 100, 3, 2000)
    want = cache.attend(table, lens, q, qr, 0.06)
    graphs, outs = [], []
    for i in range(2):  # each has its own workspace
        graph, out = torch.cuda.CUDAGraph(), torch.empty_like(q)
        with torch.cuda.graph(graph):
            cache.attend(table, lens, q, qr, 0.06, out=out)
        graphs.append(graph)
        outs.append(out)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for out in outs)
    lens.copy_(ints(5760, 1, 0, 2001))  # a captured call keeps working as lengths grow
    graphs[0].replay()
    assert torch.equal(outs[0], cache.attend(table, lens, q, qr, 0.06))
    got = cache.attend(table, lens, q, qr, 0.06, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(got, outs[0])
    for _ in range(10):
        assert torch.equal(cache.attend(table, lens, q, qr, 0.06), got)


@gpu
def test_the_bindings_refusals():
    cache = make_cache(torch.bfloat16, 10, 16)
    table = make_table(2, 4, 10)
    q, qr = queries(torch.bfloat16, 2, 1, 16)
    lens = ints(10, 20)
    good = dict(table=table, lens=lens, q=q, q_rope=qr, scale=0.1)
    for over in (dict(table=table.long()), dict(table=table[0]), dict(table=table.t()), dict(lens=None),
                 dict(lens=lens.long()), dict(lens=lens[:1]), dict(starts=lens[:1]), dict(q=q.half()), dict(q=q[..., :256]),
                 dict(q_rope=qr[..., :32]), dict(q_rope=qr.half()), dict(q_rope=qr[:, :, :5]), dict(q=q[:1]),
                 dict(out=q.half()), dict(out=q[:, :, :3]), dict(out=q[:1, :1].expand(2, 1, 16, 512)), dict(scale="x"),
                 dict(status=lens), dict(q=q.transpose(2, 3))):
        with pytest.raises(ValueError):
            cache.attend(**{**good, **over})
    with pytest.raises(mk.MKError):
        cache.attend(**{**good, "scale": math.nan})
    rows = torch.zeros((2, 3, 576), device="cuda")
    good = dict(table=table, positions=lens, rows=rows)
    for over in (dict(positions=None), dict(positions=lens.long()), dict(rows=rows.double()), dict(rows=rows[..., :570]),
                 dict(rows=rows[:1]), dict(rows=rows[0]), dict(counts=lens[:1]), dict(gain=torch.ones(512)),
                 dict(gain=torch.ones(500, device="cuda")), dict(gain=lens), dict(inv_freq=torch.ones(32, device="cuda")),
                 dict(inv_freq=rotary.frequencies(64), layout="no"), dict(eps="x"), dict(magnitude="x"),
                 dict(rows=rows.transpose(1, 2))):
        with pytest.raises(ValueError):
            cache.write(**{**good, **over})
    with pytest.raises(mk.MKError):
        cache.write(**{**good, "inv_freq": rotary.frequencies(32)})
    x = torch.zeros((4, 16, 512), device="cuda", dtype=torch.bfloat16)
    for a, b in ((x.float(), x.float()), (x, x.half()), (x, x[:, :8]), (x[0], x[0]), (x.cpu(), x.cpu()),
                 (x.transpose(1, 2), x)):
        with pytest.raises(ValueError):
            latent.LatentPages(a, b)
    # nothing to do
    assert cache.attend(table[:0], lens[:0], q[:0], qr[:0], 0.1).shape == (0, 1, 16, 512)
    cache.write(table, lens, rows[:, :0])


# ---------------------------------------------------------------- together

@gpu
def test_a_step_of_attention_in_both_forms():
    """Down-projection to output: the absorbed form over the cache that write filled equals the expanded form over keys
    and values made from the same latents, and both the definition, for a prompt's last tokens."""
    B, T, H, n = 2, 3, 16, 150
    g = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    rows = normal(B, n, 576).bfloat16()
    gain, freq = (1 + 0.1 * normal(512)).bfloat16(), rotary.frequencies(64)
    w_uk, w_uv = normal(H, 128, 512) * 512 ** -0.5, normal(H, 128, 512) * 512 ** -0.5
    q = normal(B, T, H, 192).bfloat16()
    cache = make_cache(torch.bfloat16, 2 * 10, 16)
    table = make_table(B, 10, 20)
    cache.write(table, ints(0, 0), rows, gain=gain, inv_freq=freq)
    q_rope = rotary.rotate(q[..., 128:], ints(n - T, n - T), freq)
    q_lat = torch.einsum("bthd,hdr->bthr", q[..., :128].float(), w_uk).bfloat16()
    lens = ints(n, n)
    o_lat, lse = cache.attend(table, lens, q_lat, q_rope, 192 ** -0.5, return_lse=True)
    out = torch.einsum("bthr,hdr->bthd", o_lat.float(), w_uv)
    # the definition from the cached values, in 64 bits, without absorbing
    at = torch.arange(n, device="cuda")
    c, r = (x[table[:, at // 16].long(), at % 16].double() for x in (cache.latent, cache.rope))
    k = torch.einsum("bnr,hdr->bnhd", c, w_uk.double())
    v = torch.einsum("bnr,hdr->bnhd", c, w_uv.double())
    x = torch.einsum("bthd,bnhd->bhtn", q[..., :128].double(), k) + torch.einsum("bthd,bnd->bhtn", q_rope.double(), r)
    x = (x * 192 ** -0.5).masked_fill(at > n - T + torch.arange(T, device="cuda")[:, None], -math.inf)
    want = torch.einsum("bhtn,bnhd->bthd", torch.softmax(x, -1), v)
    # the absorbed query is rounded to bf16 (2^-8 of its 512 values, whose errors add like a random walk), the weights
    # and the latent outputs too: an order of 2^-8 each of values of order 1
    assert (out.double() - want).abs().max() < 8 * 2.0 ** -8
    assert (lse.double().transpose(1, 2) - torch.logsumexp(x, -1)).abs().max() < 8 * 2.0 ** -8
    kb, vb = k.bfloat16().reshape(B * n, H, 128), v.bfloat16().reshape(B * n, H, 128)
    got = latent.attend_prompt(torch.cat([q[..., :128], q_rope], -1).reshape(B * T, H, 192), kb,
                               r.bfloat16().reshape(B * n, 64), vb, ints(0, T, 2 * T), ints(0, n, 2 * n), 192 ** -0.5)
    assert (got.double().view(B, T, H, 128) - want).abs().max() < 8 * 2.0 ** -8


@gpu
def test_a_models_own_cache():
    """The decode step's latent cache through latent_pages: what kv.read gives, attended to, and written to."""
    from moe_decode_megakernel_02_gb300 import workload
    from synth import configs
    cfg = configs.scaled(configs.DEEP, n_layers=2, n_routed_experts=8, top_k=2, vocab=1024)
    model = workload.load_synthetic(cfg, max_batch=2, max_tokens_per_seq=1, max_ctx=200)
    kv = mk.KVCache(model, 2, 200)
    workload.prefill(kv, cfg, 150)
    with pytest.raises(mk.MKError):
        kv.latent_pages(2)
    for layer in (0, 1):
        cache = kv.latent_pages(layer)
        assert cache.rank == 512 and cache.rope_dim == 64 and cache.table.shape[0] == 2
        for b in range(2):
            rows = torch.from_numpy(kv.read(layer, b, 0, 150).view("int16")).cuda().view(torch.bfloat16)
            at = torch.arange(150, device="cuda")
            page, row = cache.table[b, at // 64].long(), at % 64
            assert torch.equal(cache.latent[page, row], rows[:, :512]) and torch.equal(cache.rope[page, row], rows[:, 512:])
    q, qr = queries(torch.bfloat16, 2, 1, 16)
    check_attend(cache, cache.table, ints(150, 77), q, qr, 192 ** -0.5)
    x = torch.randn((2, 4, 576), device="cuda").bfloat16()
    cache.write(cache.table, ints(150, 150), x)
    torch.cuda.synchronize()
    got = torch.from_numpy(kv.read(1, 1, 150, 4).view("int16")).cuda().view(torch.bfloat16)
    assert torch.equal(got, x[1])
