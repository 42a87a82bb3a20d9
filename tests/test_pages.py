"""Paged caches of the caller: quantising writes, reads, and attention over the pages.

CPU: the refusals of the C entry points and of the binding. GPU: every format
against the definition in 64 bits, at the sizes and masks where a kernel can go
wrong; what a call must leave alone; the operators in a row.

Tolerances. Codes: the kernel's 32-bit quotients are correctly rounded, so codes
and scales equal the ones torch computes with true 32-bit divisions, bit for bit.
Reading rounds code x scale once to 32 bits and once to the output type: 2^-24 +
eps/2 of the value. Attention: a score is a sum of D products, exact in 32 bits
each, whose sum and scaling lose at most about (D + 8) 2^-24 of sum |q k| scale;
e^x turns that absolute error into a relative one of every weight, softmax
normalises (a factor 2). Probabilities keep 16 bits (bf16 pages, hi + lo: 2^-8 of
what 2^-8 left) or 11 (8-bit pages: half a step of fp16, 2^-11, and for the smallest
half of fp16's least step, 2^-25, where 2^15 stands for up to twice the largest V
scale: 2^-39 of the largest possible |v| each), 32-bit sums of L weights add less than 2^-20, and the
result is rounded to its type, eps/2 of the value. The bound below sums these
against sum_j p_j |v_j|.
"""
import ctypes
import math

import pytest
import torch

import moe_decode_megakernel_02_gb300 as mk
from moe_decode_megakernel_02_gb300 import pages

gpu = pytest.mark.gpu
QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}
FORMATS = [torch.bfloat16, torch.float8_e4m3fn, torch.int8]


def quantised(x, dtype):
    """Codes and scales by true 32-bit divisions."""
    x = x.float()
    if dtype == torch.bfloat16:
        return x.to(dtype), None
    a = x.abs().amax(-1)
    s = (a / torch.full_like(a, QMAX[dtype])).clamp_min(2.0 ** -126)
    y = x / s[..., None]
    return (y.round().to(dtype) if dtype == torch.int8 else y.to(dtype)), s


def make_cache(dtype, n, H, ps, D, seed=0, fill=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((2, n, H, ps, D), generator=g, device="cuda")
    (k, ks), (v, vs) = (quantised(x[i] if fill else 0 * x[i], dtype) for i in (0, 1))
    return pages.Pages(k.contiguous(), v.contiguous(), ks, vs)


def values(c, s):
    """64-bit values of a cache plane [n, H, ps, D]."""
    return c.double() if s is None else c.double() * s.double()[..., None]


def make_table(B, cols, n, seed=0, shared=0):
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(n, generator=g)
    t = torch.empty((B, cols), dtype=torch.int32)
    t[:, :shared] = order[:shared]
    t[:, shared:] = order[shared:shared + B * (cols - shared)].view(B, -1)
    return t.cuda()


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- refusals (CPU)

def _structs(**over):
    one = 4096  # an address that is aligned and never followed
    p = dict(k=one, v=one, k_scale=None, v_scale=None, page_stride=4 * 64 * 64, head_stride=64 * 64, row_stride=64,
             scale_page_stride=0, scale_head_stride=0, format=mk.KV_BF16, n_pages=8, n_kv_heads=4, page_size=64,
             head_dim=64, reserved=0)
    t = dict(table=one, stride=4, batch=2, pages_per_seq=4)
    r = dict(data=one, seq_stride=256, token_stride=256, head_stride=64, dtype=mk.DT_BF16, reserved=0)
    a = dict(lens=one, starts=None, slopes=None, lse=None, status=None, n_tokens=1, n_q_heads=8, scale=0.125,
             softcap=0.0, shared_len=0, reserved=0)
    for key, val in over.items():
        group, name = key.split("__")
        {"p": p, "t": t, "r": r, "a": a}[group][name] = val
    return mk.PagesStruct(**p), mk.TableStruct(**t), mk.RowsStruct(**r), a


BAD_PAGES = [
    (dict(p__k=None), mk.ERR_INVALID_ARG), (dict(p__format=3), mk.ERR_INVALID_ARG),
    (dict(p__format=mk.KV_E4M3), mk.ERR_INVALID_ARG), (dict(p__k_scale=4096, p__v_scale=4096), mk.ERR_INVALID_ARG),
    (dict(p__head_dim=60), mk.ERR_UNSUPPORTED), (dict(p__head_dim=264), mk.ERR_UNSUPPORTED),
    (dict(p__head_dim=0), mk.ERR_INVALID_ARG), (dict(p__page_size=48), mk.ERR_UNSUPPORTED),
    (dict(p__page_size=0), mk.ERR_UNSUPPORTED), (dict(p__n_pages=0), mk.ERR_INVALID_ARG),
    (dict(p__k=4104), mk.ERR_INVALID_ARG), (dict(p__row_stride=68), mk.ERR_INVALID_ARG),
    (dict(p__page_stride=-64), mk.ERR_INVALID_ARG), (dict(t__batch=0), mk.ERR_INVALID_ARG),
    (dict(t__pages_per_seq=0), mk.ERR_INVALID_ARG), (dict(t__table=None), mk.ERR_INVALID_ARG),
    (dict(t__stride=-1), mk.ERR_INVALID_ARG), (dict(t__pages_per_seq=1 << 25), mk.ERR_UNSUPPORTED),
    (dict(r__data=None), mk.ERR_INVALID_ARG), (dict(r__dtype=7), mk.ERR_INVALID_ARG),
    (dict(r__data=4097), mk.ERR_INVALID_ARG),
]


@pytest.mark.parametrize("over,code", BAD_PAGES)
def test_bad_pages_are_refused(over, code):
    p, t, r, a = _structs(**over)
    ref = ctypes.byref
    L = mk.lib()
    for f in (L.mk_pages_write, L.mk_pages_read):
        assert f(ref(p), ref(t), 4096, None, 1, ref(r), ref(r), None, None) == code
        assert L.mk_last_error()
    if not any(k.startswith("r__dtype") for k in over):
        att = mk.AttentionStruct(pages=ctypes.pointer(p), table=ctypes.pointer(t), q=ctypes.pointer(r),
                                 out=ctypes.pointer(r), **a)
        assert L.mk_pages_attend(ref(att), 4096, 1 << 30, None) == code


def test_null_and_negative_counts_are_refused():
    p, t, r, a = _structs()
    ref, L = ctypes.byref, mk.lib()
    assert L.mk_pages_write(None, ref(t), 4096, None, 1, ref(r), ref(r), None, None) == mk.ERR_INVALID_ARG
    assert L.mk_pages_write(ref(p), None, 4096, None, 1, ref(r), ref(r), None, None) == mk.ERR_INVALID_ARG
    assert L.mk_pages_write(ref(p), ref(t), None, None, 1, ref(r), ref(r), None, None) == mk.ERR_INVALID_ARG
    assert L.mk_pages_write(ref(p), ref(t), 4096, None, -1, ref(r), ref(r), None, None) == mk.ERR_INVALID_ARG
    assert L.mk_pages_write(ref(p), ref(t), 4096, None, 1, None, ref(r), None, None) == mk.ERR_INVALID_ARG
    r2 = _structs(r__dtype=mk.DT_F16)[2]
    assert L.mk_pages_write(ref(p), ref(t), 4096, None, 1, ref(r), ref(r2), None, None) == mk.ERR_INVALID_ARG
    assert L.mk_pages_write(ref(p), ref(t), 4096, None, 0, ref(r), ref(r), None, None) == mk.OK  # nothing to do
    assert L.mk_pages_attend(None, 4096, 1 << 30, None) == mk.ERR_INVALID_ARG
    assert L.mk_pages_attend_workspace(None, None) == mk.ERR_INVALID_ARG
    assert L.mk_kv_view(None, 0, ref(p), ref(t)) == mk.ERR_INVALID_ARG


@pytest.mark.parametrize("over,code", [
    (dict(p__head_dim=96, p__row_stride=96), mk.ERR_UNSUPPORTED), (dict(a__n_tokens=0), mk.ERR_INVALID_ARG),
    (dict(a__n_q_heads=6), mk.ERR_INVALID_ARG), (dict(a__n_q_heads=0), mk.ERR_INVALID_ARG),
    (dict(a__lens=None), mk.ERR_INVALID_ARG), (dict(r__dtype=mk.DT_F32), mk.ERR_INVALID_ARG),
    (dict(a__softcap=-1.0), mk.ERR_INVALID_ARG), (dict(a__softcap=math.nan), mk.ERR_INVALID_ARG),
    (dict(a__scale=math.nan), mk.ERR_INVALID_ARG), (dict(a__shared_len=32), mk.ERR_INVALID_ARG),
    (dict(a__shared_len=-64), mk.ERR_INVALID_ARG), (dict(a__shared_len=64 * 5), mk.ERR_INVALID_ARG),
    (dict(p__k=4096 + 8, p__v=4096 + 8, p__format=mk.KV_INT8, p__k_scale=4096, p__v_scale=4096), mk.ERR_INVALID_ARG),
    (dict(p__row_stride=72, p__format=mk.KV_INT8, p__k_scale=4096, p__v_scale=4096), mk.ERR_INVALID_ARG),
])
def test_bad_attention_arguments_are_refused(over, code):
    p, t, r, a = _structs(**over)
    att = mk.AttentionStruct(pages=ctypes.pointer(p), table=ctypes.pointer(t), q=ctypes.pointer(r),
                             out=ctypes.pointer(r), **a)
    assert mk.lib().mk_pages_attend(ctypes.byref(att), 4096, 1 << 30, None) == code
    n = ctypes.c_int64()
    assert mk.lib().mk_pages_attend_workspace(ctypes.byref(att), ctypes.byref(n)) == code


# ---------------------------------------------------------------- write and read

@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B,T,H,D,ps", [(1, 1, 1, 64, 16), (3, 37, 2, 128, 16), (2, 130, 3, 80, 64), (5, 9, 4, 256, 1),
                                        (2, 70, 1, 8, 32)])
def test_write_and_read_match_the_definition(dtype, fmt, B, T, H, D, ps):
    g = torch.Generator(device="cuda").manual_seed(B * T + D)
    cols = -(-(T + 11) // ps)
    n = B * cols + 2
    cache = make_cache(fmt, n, H, ps, D, seed=1)
    before = [x.clone() if x is not None else None for x in (cache.k, cache.k_scale, cache.v, cache.v_scale)]
    table = make_table(B, cols, n)
    pos = torch.randint(0, 12, (B,), generator=g, device="cuda").to(torch.int32)
    counts = torch.randint(0, T + 1, (B,), generator=g, device="cuda").to(torch.int32)
    new = (torch.randn((B, T, 2, H, D), generator=g, device="cuda") * 3).to(dtype)
    status = ints(0)
    cache.write(table, pos, new[:, :, 0], new[:, :, 1], counts=counts, status=status)
    want = [x.clone() if x is not None else None for x in before]
    for b in range(B):
        for t in range(int(counts[b])):
            j = int(pos[b]) + t
            pg, r = int(table[b, j // ps]), j % ps
            for i in (0, 1):
                c, s = quantised(new[b, t, i], fmt)
                want[2 * i][pg, :, r] = c
                if s is not None:
                    want[2 * i + 1][pg, :, r] = s
    for got, w in zip((cache.k, cache.k_scale, cache.v, cache.v_scale), want):
        if w is not None:
            raw = torch.uint8 if w.dtype == torch.float8_e4m3fn else w.dtype
            assert torch.equal(got.view(raw), w.view(raw))
    # and back, in another type; rows past the counts stay
    back = torch.full((2, B, T, H, D), -7.0, device="cuda").to(dtype)
    cache.read(table, pos, back[0], back[1], counts=counts, status=status)
    eps = 2.0 ** -24 + torch.finfo(dtype).eps / 2
    for i, (c, s) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        whole = values(c, s)
        for b in range(B):
            m = int(counts[b])
            assert bool((back[i, b, m:] == -7).all())
            if m:
                j = int(pos[b]) + torch.arange(m, device="cuda")
                ref = whole[table[b, j // ps].long(), :, j % ps]
                # below a type's normal range its step is absolute
                tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
                assert bool(((back[i, b, :m].double() - ref).abs() <= eps * ref.abs() + tiny).all())
    assert int(status) == 0


@gpu
@pytest.mark.parametrize("fmt", FORMATS[1:])
def test_rows_at_the_ends_of_the_range(fmt):
    """Zeros, the least and the largest numbers, and every rounding tie of a row."""
    D = 256
    rows = torch.zeros((1, 8, 1, D), device="cuda")
    rows[0, 1] = 2.0 ** -149
    rows[0, 2, 0, ::2] = torch.finfo(torch.float32).max
    rows[0, 2, 0, 1::2] = -torch.finfo(torch.float32).max
    rows[0, 3] = torch.linspace(-127, 127, D, device="cuda") * 2.0 ** -100
    rows[0, 4] = (torch.arange(D, device="cuda") - 127.5).clamp(-127, 127)  # int8: ties everywhere
    rows[0, 5] = torch.linspace(0, 448, D, device="cuda").round()
    rows[0, 6] = torch.linspace(-1, 1, D, device="cuda") * 2.0 ** -126
    rows[0, 7] = torch.randn(D, device="cuda") * 1e30
    cache = make_cache(fmt, 1, 1, 8, D, fill=False)
    cache.write(ints(0).view(1, 1), ints(0), rows, rows)
    c, s = quantised(rows[0, :, 0], fmt)
    # code x scale stays finite: the scale is held at the largest number over the format's
    s = torch.minimum(s, torch.tensor({torch.float8_e4m3fn: 448, torch.int8: 127}[fmt], device="cuda").double().pow(-1)
                      .mul(torch.finfo(torch.float32).max).float())
    assert torch.allclose(cache.k_scale[0, 0], s, rtol=2.0 ** -22, atol=0)
    ok = torch.tensor([0, 1, 3, 4, 5, 6, 7], device="cuda")
    raw = torch.uint8 if fmt == torch.float8_e4m3fn else fmt
    assert torch.equal(cache.k[0, 0][ok].view(raw), c[ok].view(raw))
    back = torch.empty((2, 1, 8, 1, D), device="cuda")
    cache.read(ints(0).view(1, 1), ints(0), back[0], back[1])
    assert bool(torch.isfinite(back).all())
    big = back[0, 0, 2, 0] / rows[0, 2, 0]
    assert bool(((big - 1).abs() < 2.0 ** -20).all())


@gpu
@pytest.mark.parametrize("fmt", FORMATS[1:])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_row_with_a_non_finite_value_reads_back_as_nan(fmt, bad):
    x = torch.randn((1, 4, 2, 64), device="cuda")
    y = x.clone()
    x[0, 2, 1, 17] = bad
    cache = make_cache(fmt, 1, 2, 4, 64)
    cache.write(ints(0).view(1, 1), ints(0), x, y)
    k, v = (torch.empty_like(x) for _ in range(2))
    cache.read(ints(0).view(1, 1), ints(0), k, v)
    nan = torch.zeros((1, 4, 2, 64), dtype=torch.bool, device="cuda")
    nan[0, 2, 1] = True
    assert torch.equal(torch.isnan(k), nan) and not bool(torch.isnan(v).any())


@gpu
def test_odd_strides_and_alignment_give_the_same_codes():
    B, T, H, D = 2, 5, 3, 64
    x = torch.randn((B, T, 2, H, D), device="cuda").to(torch.bfloat16)
    wide = torch.empty((H, T, B, D + 3), dtype=torch.bfloat16, device="cuda")[..., 1:D + 1].permute(2, 1, 0, 3)
    wide.copy_(x[:, :, 0])
    table = make_table(B, 2, 4)
    a, b = (make_cache(torch.int8, 4, H, 8, D, fill=False) for _ in range(2))
    a.write(table, ints(1, 3), x[:, :, 0], x[:, :, 1])
    b.write(table, ints(1, 3), wide, x[:, :, 1])
    assert torch.equal(a.k, b.k) and torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v, b.v)
    got = torch.zeros_like(wide)
    got2 = torch.empty((H, T, B, D + 3), dtype=torch.bfloat16, device="cuda")[..., 1:D + 1].permute(2, 1, 0, 3)
    got = torch.empty_like(x[:, :, 0].contiguous())
    a.read(table, ints(1, 3), got, torch.empty_like(got))
    a.read(table, ints(1, 3), got2, torch.empty_like(got))
    assert torch.equal(got, got2)


@gpu
def test_positions_and_pages_out_of_range_are_skipped_and_reported():
    cache = make_cache(torch.int8, 2, 1, 4, 64, fill=False)
    x = torch.ones((3, 3, 1, 64), device="cuda", dtype=torch.bfloat16)
    table = torch.tensor([[0, 5], [-1, 1], [1, 0]], dtype=torch.int32, device="cuda")
    status = ints(0)
    # sequence 0: row 3 of page 0, then page 5; sequence 1: page -1, then page 1; sequence 2: past the table
    cache.write(table, ints(3, 3, 8), x, x, status=status)
    assert int(status) == mk.ERR_INVALID_ARG
    want = torch.zeros((2, 1, 4), dtype=torch.bool, device="cuda")
    want[0, 0, 3] = want[1, 0, 0] = want[1, 0, 1] = True
    assert torch.equal(cache.k[..., 0] != 0, want)
    status.zero_()
    cache.write(table, ints(-2, 0, -1), x, x, counts=ints(2, 0, 1), status=status)
    assert int(status) == mk.ERR_INVALID_ARG
    assert torch.equal(cache.k[..., 0] != 0, want)
    status.zero_()
    out = torch.full_like(x, 9)
    cache.read(table, ints(3, 3, 8), out, torch.empty_like(out), status=status)
    assert int(status) == mk.ERR_INVALID_ARG
    assert (out[..., 0, 0] != 9).tolist() == [[True, False, False], [False, True, True], [False] * 3]


# ---------------------------------------------------------------- attention

def reference(cache, table, lens, q, scale, softcap=0.0, slopes=None, starts=None):
    """Output, lse and sum_j p_j |v_j| in 64 bits, sum of |q k| scale bounds included."""
    B, T, Hq, D = q.shape
    n, H, ps, _ = cache.k.shape
    K, V = values(cache.k, cache.k_scale), values(cache.v, cache.v_scale)
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device="cuda")
    mag, lse = torch.zeros_like(out), torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    reach = torch.zeros((B, T, Hq), dtype=torch.float64, device="cuda")
    for b in range(B):
        L = int(lens[b])
        for t in range(T):
            p = L - T + t
            lo = int(starts[b]) if starts is not None else 0
            if p < lo or p < 0:
                continue
            j = torch.arange(max(lo, 0), p + 1, device="cuda")
            pg, r = table[b, j // ps].long(), j % ps
            k, v = K[pg, :, r], V[pg, :, r]  # [L, H, D]
            qq = q[b, t].double().view(H, Hq // H, D)
            x = torch.einsum("hgd,lhd->hgl", qq, k) * scale
            reach[b, t] = (torch.einsum("hgd,lhd->hgl", qq.abs(), k.abs()) * abs(scale)).amax(-1).reshape(-1)
            if softcap > 0:
                x = softcap * torch.tanh(x / softcap)
            x = x.reshape(Hq, -1)
            if slopes is not None:
                x = x - slopes.double()[:, None] * (p - j).double()
            w = torch.softmax(x, -1).view(H, Hq // H, -1)
            out[b, t] = torch.einsum("hgl,lhd->hgd", w, v).reshape(Hq, D)
            mag[b, t] = torch.einsum("hgl,lhd->hgd", w, v.abs()).reshape(Hq, D)
            lse[b, t] = torch.logsumexp(x, -1)
    return out, lse, mag, reach


def check(cache, table, lens, q, out, lse, scale, **kw):
    ref, rlse, mag, reach = reference(cache, table, lens, q, scale, **kw)
    D = q.shape[-1]
    cap = kw.get("softcap", 0.0)
    far = 0.0
    if kw.get("slopes") is not None:  # the bias is one rounded product of up to slope * L
        far = float(kw["slopes"].max()) * float(lens.max())
    # absolute error of a score: products' sum, scaling and log2 e (8 roundings), the cap's 4 steps of its size
    dx = (D + 8) * 2.0 ** -24 * (reach + far + 1) + 4 * cap * 2.0 ** -23 + 2.0 ** -20
    weight = 2 * dx + (2.0 ** -16 if cache.k.dtype == torch.bfloat16 else 2.0 ** -11)
    eps = torch.finfo(q.dtype).eps / 2
    tiny = torch.finfo(q.dtype).smallest_normal * torch.finfo(q.dtype).eps
    if cache.k.dtype != torch.bfloat16:
        tiny += float(lens.max()) * 2.0 ** -39 * QMAX[cache.k.dtype] * float(cache.v_scale[cache.v_scale < 1e6].max())
    bound = weight[..., None] * mag + eps * (ref.abs() + weight[..., None] * mag) + tiny
    d = (out.double() - ref).abs()
    worst = float((d - bound).max())
    assert worst <= 0, f"off by {float(d.max()):.3g}, {float((d / bound.clamp_min(1e-30)).max()):.3g} of the bound"
    empty = rlse == -math.inf
    assert bool((lse[empty] == -math.inf).all()) and bool((out[empty] == 0).all())
    assert bool(((lse.double() - rlse).abs()[~empty] <= (dx + 2.0 ** -22 * rlse.abs())[~empty]).all())


def build(fmt, qdtype, B, T, Hq, H, D, ps, lens, shared=0, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cols = max(1, -(-max(lens) // ps)) + 1
    sp = shared // ps
    n = sp + B * (cols - sp) + 1
    cache = make_cache(fmt, n, H, ps, D, seed=seed)
    table = make_table(B, cols, n, shared=sp)
    q = (torch.randn((B, T, Hq, D), generator=g, device="cuda") * 1.5).to(qdtype)
    return cache, table, ints(*lens), q


@gpu
@pytest.mark.parametrize("qdtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B,T,Hq,H,D,ps,lens", [
    (1, 1, 1, 1, 64, 16, [1]),                      # one position
    (1, 1, 4, 4, 128, 64, [64]),                    # no groups, a whole tile
    (3, 1, 16, 4, 128, 64, [0, 65, 1000]),          # an empty sequence
    (2, 7, 16, 4, 128, 64, [5, 700]),               # fewer positions than tokens; 28 rows
    (2, 7, 40, 8, 64, 16, [300, 129]),              # 35 rows
    (4, 1, 24, 1, 128, 32, [257, 3, 511, 1]),       # 24 rows on one kv head
    (2, 5, 8, 2, 256, 128, [390, 77]),              # 20 rows of 256
    (1, 33, 6, 2, 64, 1, [200]),                    # 99 rows, pages of one position
    (37, 1, 5, 1, 64, 16, list(range(37))),         # many short sequences
])
def test_attention_matches_the_definition(qdtype, fmt, B, T, Hq, H, D, ps, lens):
    cache, table, n, q = build(fmt, qdtype, B, T, Hq, H, D, ps, lens)
    scale = 1 / math.sqrt(D)
    status = ints(0)
    out, lse = cache.attend(table, n, q, return_lse=True, status=status)
    check(cache, table, n, q, out, lse, scale)
    assert int(status) == 0
    assert torch.equal(cache.attend(table, n, q), out)  # the same call again, without lse


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kw", [dict(softcap=20.0), dict(slopes=True), dict(starts=True),
                                dict(softcap=50.0, slopes=True, starts=True)])
def test_caps_biases_and_document_starts(fmt, D, kw):
    B, T, Hq, H = 3, 2, 10, 2
    cache, table, n, q = build(fmt, torch.bfloat16, B, T, Hq, H, D, 32, [333, 64, 1500])
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = torch.exp2(-torch.arange(1, Hq + 1, device="cuda").float())
    if kw.get("starts"):
        kw["starts"] = ints(100, 63, 1600)  # inside; the last token alone; past the end: empty rows
    out, lse = cache.attend(table, n, q, scale=0.3, return_lse=True, **kw)
    check(cache, table, n, q, out, lse, 0.3, **kw)


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B,T,Hq,H,D,ps,shared,lens", [
    (3, 1, 8, 2, 128, 64, 640, [641, 640, 900]),
    (9, 1, 40, 8, 128, 16, 208, [300, 0, 209, 999, 208, 215, 256, 257, 1000]),  # a padded sequence among them
    (5, 4, 4, 4, 64, 16, 16, [20, 36, 16, 100, 18]),
    (2, 7, 8, 1, 256, 32, 320, [327, 700]),
    (33, 3, 4, 1, 64, 64, 128, [131 + i for i in range(33)]),                   # 396 rows on one head
])
def test_a_shared_prefix_gives_what_separate_pages_give(fmt, B, T, Hq, H, D, ps, shared, lens):
    cache, table, n, q = build(fmt, torch.bfloat16, B, T, Hq, H, D, ps, lens, shared=shared)
    scale = 1 / math.sqrt(D)
    out, lse = cache.attend(table, n, q, shared_len=shared, return_lse=True)
    check(cache, table, n, q, out, lse, scale)
    plain, plse = cache.attend(table, n, q, return_lse=True)
    check(cache, table, n, q, plain, plse, scale)
    kw = dict(softcap=30.0, slopes=torch.full((Hq,), 0.01, device="cuda"),
              starts=ints(*[7 * (b % 3) * shared // 16 for b in range(B)]))
    out, lse = cache.attend(table, n, q, shared_len=shared, return_lse=True, **kw)
    check(cache, table, n, q, out, lse, scale, **kw)


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shared", [0, 32])
def test_what_a_row_does_not_see_cannot_reach_it(fmt, shared):
    """NaN and infinities past the end, before the start, in later tokens and in unused pages."""
    B, T, Hq, H, D, ps = 2, 3, 4, 2, 64, 16
    lens = [70, 41]
    cache, table, n, q = build(fmt, torch.bfloat16, B, T, Hq, H, D, ps, lens, shared=shared)
    starts = ints(9, 0)
    clean, clse = cache.attend(table, n, q, starts=starts, shared_len=shared, return_lse=True)
    seen = torch.zeros((cache.k.shape[0], ps), dtype=torch.bool, device="cuda")
    for b in range(B):
        for j in range(int(starts[b]), lens[b]):
            seen[table[b, j // ps].long(), j % ps] = True
    hide = (~seen)[:, None, :].expand(-1, H, -1)
    if fmt == torch.bfloat16:
        cache.k[hide], cache.v[hide] = math.nan, math.inf
    else:
        cache.k_scale[hide], cache.v_scale[hide] = math.nan, math.inf
        if fmt == torch.float8_e4m3fn:
            cache.v.view(torch.uint8)[hide] = 0x7F
    out, lse = cache.attend(table, n, q, starts=starts, shared_len=shared, return_lse=True)
    assert torch.equal(out, clean) and torch.equal(lse, clse)
    # the last token's own values: the earlier tokens must not see them, the last one must
    for b in range(B):
        j = lens[b] - 1
        pg, r = int(table[b, j // ps]), j % ps
        if fmt == torch.int8:
            cache.v_scale[pg, :, r] = math.nan
        elif fmt == torch.bfloat16:
            cache.v[pg, :, r] = math.nan
        else:
            cache.v.view(torch.uint8)[pg, :, r] = 0x7F
    out, lse = cache.attend(table, n, q, starts=starts, shared_len=shared, return_lse=True)
    assert torch.equal(out[:, :-1], clean[:, :-1]) and torch.equal(lse[:, :-1], clse[:, :-1])
    assert bool(torch.isnan(out[:, -1]).all())


@gpu
def test_infinite_values_that_are_seen_stay_infinite():
    cache, table, n, q = build(torch.bfloat16, torch.bfloat16, 1, 2, 4, 2, 64, 16, [40])
    pg = int(table[0, 2])
    cache.v[pg, :, 6, 5] = math.inf  # position 38: seen by both tokens
    cache.v[pg, :, 7, 9] = -math.inf  # position 39: by the last
    out = cache.attend(table, n, q)
    assert bool((out[0, :, :, 5] == math.inf).all())
    assert bool((out[0, 1, :, 9] == -math.inf).all()) and bool(torch.isfinite(out[0, 0, :, 9]).all())
    rest = [d for d in range(64) if d not in (5, 9)]
    assert bool(torch.isfinite(out[..., rest]).all())


@gpu
def test_lengths_and_pages_out_of_range_are_reported_and_stay_inside():
    cache, table, n, q = build(torch.bfloat16, torch.bfloat16, 2, 1, 4, 2, 64, 16, [40, 40])
    status = ints(0)
    cache.attend(table, ints(40, 16 * table.shape[1] + 1), q, status=status)
    assert int(status) == mk.ERR_INVALID_ARG
    status.zero_()
    bad = table.clone()
    bad[1, 1] = cache.k.shape[0]
    bad[0, 0] = -5
    out = cache.attend(bad, n, q, status=status)
    assert int(status) == mk.ERR_INVALID_ARG and bool(torch.isfinite(out).all())
    status.zero_()
    out, lse = cache.attend(table, ints(-3, -2147483648), q, status=status, return_lse=True)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all()) and int(status) == 0


@gpu
def test_strided_queries_outputs_caches_and_tables():
    B, T, Hq, H, D, ps = 2, 3, 8, 2, 128, 16
    cache, table, n, q = build(torch.float8_e4m3fn, torch.bfloat16, B, T, Hq, H, D, ps, [90, 33])
    want = cache.attend(table, n, q)
    n_pages = cache.k.shape[0]
    # K and V interleaved in one buffer, pages in rows of a wider one
    buf = torch.zeros((n_pages, ps, H, 2, D + 16), dtype=torch.uint8, device="cuda")
    k, v = (buf[:, :, :, i, :D].permute(0, 2, 1, 3).view(torch.float8_e4m3fn) for i in (0, 1))
    k.view(torch.uint8).copy_(cache.k.view(torch.uint8))
    v.view(torch.uint8).copy_(cache.v.view(torch.uint8))
    sc = torch.zeros((2, H, n_pages, ps + 5), device="cuda")
    ks, vs = (sc[i].permute(1, 0, 2)[:, :, 2:2 + ps] for i in (0, 1))
    ks.copy_(cache.k_scale)
    vs.copy_(cache.v_scale)
    wide = torch.zeros((B, table.shape[1] + 3), dtype=torch.int32, device="cuda")
    wide[:, 1:1 + table.shape[1]] = table
    qw = torch.empty((Hq, B, T, D + 1), dtype=torch.bfloat16, device="cuda")[..., 1:].permute(1, 2, 0, 3)
    qw.copy_(q)
    out = torch.full((T, B, Hq, D + 3), 5.0, dtype=torch.bfloat16, device="cuda")
    got = pages.Pages(k, v, ks, vs).attend(wide[:, 1:1 + table.shape[1]], n, qw, out=out[..., 1:D + 1].permute(1, 0, 2, 3))
    assert torch.equal(got, want)
    assert bool((out[..., 0] == 5).all()) and bool((out[..., D + 1:] == 5).all())


@gpu
def test_offsets_past_32_bits():
    """A page far past 2^32 bytes of its cache."""
    H, ps, D = 1, 64, 64
    n = (1 << 32) // (ps * D) + 70
    k = torch.empty((n, H, ps, D), dtype=torch.int8, device="cuda")
    s = torch.empty((n, H, ps), device="cuda")
    cache = pages.Pages(k, k, s, s)
    small = make_cache(torch.int8, 2, H, ps, D)
    far = [n - 1, n - 3]
    for i, pg in enumerate(far):
        k[pg], s[pg] = small.k[i], small.k_scale[i]
    q = torch.randn((1, 1, 4, D), device="cuda").to(torch.bfloat16)
    got = cache.attend(ints(*far).view(1, 2), ints(100), q)
    ref = pages.Pages(small.k, small.k, small.k_scale, small.k_scale)
    assert torch.equal(got, ref.attend(ints(0, 1).view(1, 2), ints(100), q))
    x = torch.randn((1, 3, H, D), device="cuda").to(torch.bfloat16)
    cache.write(ints(*far).view(1, 2), ints(63), x, x)
    a, b = torch.empty_like(x), torch.empty_like(x)
    cache.read(ints(*far).view(1, 2), ints(63), a, b)
    assert bool(((a - x).abs() <= 2.0 ** -6 * x.abs().amax()).all())
    assert torch.equal(k[n - 1, 0, 63], quantised(x[0, 0, 0], torch.int8)[0])


@gpu
def test_other_streams_and_graphs_have_their_own_workspaces():
    cache, table, n, q = build(torch.float8_e4m3fn, torch.bfloat16, 4, 1, 16, 4, 128, 64, [900, 1, 300, 2000])
    want = cache.attend(table, n, q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [cache.attend(table, n, q, stream=side) for _ in range(3)]
    both = [cache.attend(table, n, q) for _ in range(3)]
    side.synchronize()
    assert all(torch.equal(x, want) for x in got + both)
    # two graphs replayed side by side, with lengths that change after the capture
    q2 = torch.randn_like(q)
    n1, n2, outs, graphs = n.clone(), n.clone(), [], []
    for nn, qq in ((n1, q), (n2, q2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(cache.attend(table, nn, qq))
        graphs.append(g)
    n1.copy_(ints(33, 700, 2000, 5))
    n2.copy_(ints(2000, 2, 64, 65))
    torch.cuda.synchronize()
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
    assert torch.equal(outs[0], cache.attend(table, n1, q)) and torch.equal(outs[1], cache.attend(table, n2, q2))


@gpu
def test_binding_refuses_what_does_not_fit():
    cache, table, n, q = build(torch.bfloat16, torch.bfloat16, 2, 1, 4, 2, 64, 16, [40, 40])
    with pytest.raises(ValueError):
        pages.Pages(cache.k, cache.v.half())
    with pytest.raises(ValueError):
        pages.Pages(cache.k.cpu(), cache.v.cpu())
    with pytest.raises(ValueError):
        pages.Pages(cache.k.to(torch.int8), cache.v.to(torch.int8))
    with pytest.raises(ValueError):
        pages.Pages(cache.k.transpose(2, 3), cache.v.transpose(2, 3))
    for bad in (dict(lens=n.long()), dict(lens=n[:1]), dict(q=q.float()), dict(q=q[:1]), dict(q=q[..., :32]),
                dict(table=table.long()), dict(slopes=torch.ones(3, device="cuda")), dict(starts=n.cpu()),
                dict(shared_len=8), dict(shared_len=1 << 20), dict(softcap=-1.0), dict(out=torch.empty_like(q).half()),
                dict(q=torch.empty((2, 1, 3, 64), dtype=torch.bfloat16, device="cuda"))):
        kw = dict(dict(table=table, lens=n, q=q), **bad)
        with pytest.raises((ValueError, mk.MKError)):
            cache.attend(kw.pop("table"), kw.pop("lens"), kw.pop("q"), **kw)
    x = torch.zeros((2, 1, 2, 64), device="cuda")
    for args in ((table, n, x, x.half()), (table, n, x[:1], x[:1]), (table, n.long(), x, x), (table, n, x[..., :32], x[..., :32])):
        with pytest.raises((ValueError, mk.MKError)):
            cache.write(*args)
    assert cache.attend(table[:0], n[:0], q[:0]).shape == (0, 1, 4, 64)


@gpu
def test_a_models_own_cache_is_read_in_place():
    """mk_kv_view: the operators on the pages that the decode step fills."""
    from moe_decode_megakernel_02_gb300 import workload
    from synth import configs
    cfg = configs.TINY
    ctx = cfg["ctx"]
    model = workload.load_synthetic(cfg, max_batch=2, max_tokens_per_seq=1, max_ctx=ctx + 70)
    kv = mk.KVCache(model, 2, ctx + 70)
    workload.prefill(kv, cfg, ctx)
    logits = torch.empty((2, cfg["vocab"]), dtype=torch.float32, device="cuda")
    tok = torch.from_numpy(workload.tokens(cfg, 0, 2, 1)).cuda()
    model.decode_step(kv, tok, ints(ctx, ctx), logits)
    model.check()
    H, D = cfg["n_kv_heads"], cfg["head_dim"]
    for layer in range(cfg["n_layers"]):
        view = kv.pages(layer)
        k, v = (torch.empty((2, ctx + 1, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        view.read(view.table, ints(0, 0), k, v)
        for b in range(2):
            rows = torch.from_numpy(kv.read(layer, b, 0, ctx + 1).view("int16")).cuda().view(torch.bfloat16)
            assert torch.equal(torch.cat([k[b].flatten(1), v[b].flatten(1)], 1), rows)
        q = torch.randn((2, 1, cfg["n_q_heads"], D), device="cuda").to(torch.bfloat16)
        out, lse = view.attend(view.table, ints(ctx + 1, ctx + 1), q, return_lse=True)
        check(view, view.table, ints(ctx + 1, ctx + 1), q, out, lse, 1 / math.sqrt(D))
        # the new position goes the other way: into an 8-bit cache with the model's block table
        cache = make_cache(torch.float8_e4m3fn, view.k.shape[0], H, 64, D, fill=False)
        cache.write(view.table, ints(0, 0), k, v)
        out8, lse8 = cache.attend(view.table, ints(ctx + 1, ctx + 1), q, return_lse=True)
        check(cache, view.table, ints(ctx + 1, ctx + 1), q, out8, lse8, 1 / math.sqrt(D))


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,T,Hq,H,ps,shared", [(40, 1, 2, 2, 64, 64), (17, 2, 8, 2, 32, 1984), (70, 1, 12, 3, 16, 6160)])
def test_long_shared_prefixes(fmt, D, B, T, Hq, H, ps, shared):
    """One tile, several turns of the ring, several pieces a CTA; scores that keep rising, so that maxima move late."""
    lens = [shared + T - 1 + (7 * b) % 40 for b in range(B)]
    lens[B // 2] = 0
    lens[B // 3] = shared // 2  # ends inside: read on its own
    cache, table, n, q = build(fmt, torch.bfloat16, B, T, Hq, H, D, ps, lens, shared=shared)
    rise = torch.linspace(0.1, 2.5, shared // ps, device="cuda")
    pg = table[0, :shared // ps].long()
    if fmt == torch.bfloat16:
        cache.k[pg] = (cache.k[pg].float() * rise[:, None, None, None]).to(fmt)
    else:
        cache.k_scale[pg] *= rise[:, None, None]
        cache.v_scale[pg] *= rise.flip(0)[:, None, None]
    scale = 1 / math.sqrt(D)
    status = ints(0)
    for kw in (dict(), dict(softcap=15.0, slopes=torch.linspace(0.001, 0.02, Hq, device="cuda"))):
        out, lse = cache.attend(table, n, q, shared_len=shared, return_lse=True, status=status, **kw)
        check(cache, table, n, q, out, lse, scale, **kw)
        assert torch.equal(out, cache.attend(table, n, q, shared_len=shared, **kw))
    assert int(status) == 0


@gpu
def test_non_finite_values_in_a_shared_prefix_stay_with_who_sees_them():
    B, Hq, H, D, ps, shared = 40, 4, 2, 128, 64, 192
    lens = [shared + 5 + b for b in range(B)]
    lens[3], lens[7] = 100, 0  # ends inside the prefix; padded
    for fmt in FORMATS:
        cache, table, n, q = build(fmt, torch.bfloat16, B, 1, Hq, H, D, ps, lens, shared=shared)
        clean = cache.attend(table, n, q, shared_len=shared)
        pg = int(table[0, 2])  # positions 128 .. 191
        if fmt == torch.bfloat16:
            cache.v[pg, :, 9, 40] = math.nan
        elif fmt == torch.int8:
            cache.v_scale[pg, :, 9] = math.nan
        else:
            cache.v.view(torch.uint8)[pg, :, 9, 40] = 0xFF
        out = cache.attend(table, n, q, shared_len=shared)
        assert torch.equal(out[3], clean[3]) and bool((out[7] == 0).all())
        others = [b for b in range(B) if b not in (3, 7)]
        assert bool(torch.isnan(out[others][..., 40]).all())
        if fmt != torch.int8:
            assert bool(torch.isfinite(out[others][..., :40]).all())


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("order", ["token", "interleaved", "shifted"])
def test_shared_prefixes_in_other_layouts(fmt, order):
    """Heads inside tokens, K and V in one buffer, rows wider than a head: the same result as dense pages."""
    B, Hq, H, D, ps, shared = 40, 8, 2, 128, 16, 144
    cache, table, n, q = build(fmt, torch.bfloat16, B, 1, Hq, H, D, ps, [shared + 3 + b for b in range(B)], shared=shared)
    want = cache.attend(table, n, q, shared_len=shared)
    N, raw = cache.k.shape[0], torch.uint8 if fmt != torch.bfloat16 else fmt
    if order == "token":
        k, v = (torch.zeros((N, ps, H, D), dtype=raw, device="cuda").permute(0, 2, 1, 3) for _ in range(2))
    elif order == "interleaved":
        buf = torch.zeros((H, N, ps, 2, D), dtype=raw, device="cuda")
        k, v = (buf[:, :, :, i].permute(1, 0, 2, 3) for i in (0, 1))
    else:
        buf = torch.zeros((2, N, H, ps, D + 16), dtype=raw, device="cuda")
        k, v = (buf[i, ..., 16:] for i in (0, 1))
    k.copy_(cache.k.view(raw))
    v.copy_(cache.v.view(raw))
    other = pages.Pages(k.view(fmt), v.view(fmt), cache.k_scale, cache.v_scale)
    assert torch.equal(other.attend(table, n, q, shared_len=shared), want)


# ---------------------------------------------------------------- wide calls: many rows a kv head and long tables

def widen(table, Hq, H, T, ps):
    """More columns, of no page, up to the capacity from which whole tiles have a launch of their own."""
    rows = T * Hq // H
    tiles = 2000 * 160 // (table.shape[0] * H * -(-rows // 128) * min(rows, 128)) + 1
    return torch.nn.functional.pad(table, (0, max(0, tiles * 64 // ps - table.shape[1])), value=-1).contiguous()


@gpu
@pytest.mark.parametrize("qdtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B,T,Hq,H,D,ps,lens", [
    (1, 17, 2, 1, 64, 64, [4096]),                       # whole tiles alone but for the last tokens
    (4, 1, 80, 2, 128, 16, [1024, 0, 64, 3000]),         # one token of 40 heads: a length of whole tiles has no rest
    (3, 10, 16, 4, 128, 32, [73, 2050, 10]),             # a whole tile not seen by all tokens
    (2, 66, 4, 2, 128, 64, [900, 1500]),                 # 132 rows: a second row block of four
    (90, 33, 1, 1, 64, 8, [34 + 13 * b for b in range(90)]),
    (2, 300, 4, 2, 64, 64, [1900, 200]),                 # fewer positions than tokens
])
def test_wide_calls_match_the_definition(qdtype, fmt, B, T, Hq, H, D, ps, lens):
    cache, table, n, q = build(fmt, qdtype, B, T, Hq, H, D, ps, lens)
    table = widen(table, Hq, H, T, ps)
    scale = 1 / math.sqrt(D)
    status = ints(0)
    for kw in (dict(), dict(softcap=15.0, slopes=torch.linspace(0.001, 0.02, Hq, device="cuda"),
                            starts=ints(*[(61 * b * b) % (lens[b] + 9) for b in range(B)]))):
        out, lse = cache.attend(table, n, q, return_lse=True, status=status, **kw)
        check(cache, table, n, q, out, lse, scale, **kw)
        assert torch.equal(out, cache.attend(table, n, q, **kw))
    assert int(status) == 0


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_wide_calls_keep_what_a_row_does_not_see_out(fmt):
    B, T, Hq, H, D, ps = 3, 10, 16, 4, 128, 16
    lens, first = [2000, 333, 700], ints(130, 0, 64)
    cache, table, n, q = build(fmt, torch.bfloat16, B, T, Hq, H, D, ps, lens)
    table = widen(table, Hq, H, T, ps)
    clean, clse = cache.attend(table, n, q, starts=first, return_lse=True)
    seen = torch.zeros((cache.k.shape[0], ps), dtype=torch.bool, device="cuda")
    for b in range(B):
        j = torch.arange(int(first[b]), lens[b], device="cuda")
        seen[table[b, j // ps].long(), j % ps] = True
    hide = (~seen)[:, None, :].expand(-1, H, -1)
    if fmt == torch.bfloat16:
        cache.k[hide], cache.v[hide] = math.nan, math.inf
    else:
        cache.k_scale[hide], cache.v_scale[hide] = math.nan, math.inf
        if fmt == torch.float8_e4m3fn:
            cache.v.view(torch.uint8)[hide] = 0x7F
    out, lse = cache.attend(table, n, q, starts=first, return_lse=True)
    assert torch.equal(out, clean) and torch.equal(lse, clse)
    # a value that every row of one head sees
    pg, r = int(table[0, 500 // ps]), 500 % ps
    if fmt == torch.bfloat16:
        cache.v[pg, 1, r, 40] = math.nan
    elif fmt == torch.int8:
        cache.v_scale[pg, 1, r] = math.nan
    else:
        cache.v.view(torch.uint8)[pg, 1, r, 40] = 0xFF
    out = cache.attend(table, n, q, starts=first)
    assert bool(torch.isnan(out[0, :, 4:8, 40]).all())
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[0, :, 4:8] = False
    assert torch.equal(out[keep], clean[keep])


@gpu
def test_wide_calls_report_bad_pages_and_lengths():
    B, T, Hq, H, ps = 2, 10, 16, 4, 64
    cache, table, n, q = build(torch.int8, torch.bfloat16, B, T, Hq, H, 128, ps, [1000, 900])
    table = widen(table, Hq, H, T, ps)
    want = cache.attend(table, n, q)
    status = ints(0)
    bad = table.clone()
    bad[1, 3] = cache.k.shape[0]
    out = cache.attend(bad, n, q, status=status)
    assert int(status) == mk.ERR_INVALID_ARG and torch.equal(out[0], want[0])
    status.zero_()
    out, lse = cache.attend(table, ints(1000, table.shape[1] * ps + 1), q, return_lse=True, status=status)  # past the table
    assert int(status) == mk.ERR_INVALID_ARG
    # work is cut by the tiles of all sequences, so the other one's sums are grouped in another way: the same bound
    # holds for it, not the same bits
    check(cache, table[:1], n[:1], q[:1], out[:1], lse[:1], 1 / math.sqrt(128))


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
def test_a_shared_prefix_with_fp16_queries(fmt, D):
    B, T, Hq, H, ps, shared = 19, 2, 8, 2, 32, 1984
    lens = [shared + T - 1 + (7 * b) % 40 for b in range(B)]
    lens[5], lens[6] = 0, 700
    cache, table, n, q = build(fmt, torch.float16, B, T, Hq, H, D, ps, lens, shared=shared)
    q[1] = 2.0 ** -20  # under fp16's normal range
    for kw in (dict(), dict(softcap=15.0, slopes=torch.linspace(0.001, 0.02, Hq, device="cuda"))):
        out, lse = cache.attend(table, n, q, shared_len=shared, return_lse=True, **kw)
        check(cache, table, n, q, out, lse, 1 / math.sqrt(D), **kw)


# ---------------------------------------------------------------- calls at their limits

@pytest.mark.parametrize("over,code", [
    (dict(t__table=4098), mk.ERR_INVALID_ARG), (dict(p__n_kv_heads=65536), mk.ERR_UNSUPPORTED),
    (dict(p__format=mk.KV_INT8, p__k_scale=4097, p__v_scale=4096), mk.ERR_INVALID_ARG),
])
def test_unaligned_tables_and_too_many_heads_are_refused(over, code):
    p, t, r, a = _structs(**over)
    a["n_q_heads"] = p.n_kv_heads
    ref, L = ctypes.byref, mk.lib()
    for f in (L.mk_pages_write, L.mk_pages_read):
        assert f(ref(p), ref(t), 4096, None, 1, ref(r), ref(r), None, None) == code
    att = mk.AttentionStruct(pages=ctypes.pointer(p), table=ctypes.pointer(t), q=ctypes.pointer(r), out=ctypes.pointer(r),
                             **a)
    assert L.mk_pages_attend(ref(att), 4096, 1 << 30, None) == code


def test_unaligned_positions_and_lengths_are_refused():
    p, t, r, a = _structs()
    ref, L = ctypes.byref, mk.lib()
    for args in ((4097, None, None), (4096, 4098, None), (4096, None, 4099)):
        pos, cnt, st = args
        assert L.mk_pages_write(ref(p), ref(t), pos, cnt, 1, ref(r), ref(r), st, None) == mk.ERR_INVALID_ARG
    for name in ("lens", "starts", "slopes", "lse", "status"):
        b = dict(a, **{name: 4098})
        att = mk.AttentionStruct(pages=ctypes.pointer(p), table=ctypes.pointer(t), q=ctypes.pointer(r),
                                 out=ctypes.pointer(r), **b)
        assert L.mk_pages_attend(ref(att), 4096, 1 << 30, None) == mk.ERR_INVALID_ARG


@gpu
@pytest.mark.parametrize("D,qdtype", [(128, torch.bfloat16), (64, torch.float16), (256, torch.bfloat16)])
def test_a_padded_sequence_leads_to_no_shared_page(D, qdtype):
    """The first sequences' table rows hold no pages: the others' shared positions are found all the same."""
    B, Hq, H, ps, shared = 36, 4, 2, 16, 320
    lens = [0, 0] + [shared + 3 + b for b in range(B - 2)]
    cache, table, n, q = build(torch.int8, qdtype, B, 1, Hq, H, D, ps, lens, shared=shared)
    table[:2] = -1
    status = ints(0)
    out, lse = cache.attend(table, n, q, shared_len=shared, return_lse=True, status=status)
    check(cache, table, n, q, out, lse, 1 / math.sqrt(D))
    # nobody takes part: nothing shared is read
    n.zero_()
    out, lse = cache.attend(torch.full_like(table, -1), n, q, shared_len=shared, return_lse=True, status=status)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all()) and int(status) == 0


@gpu
@pytest.mark.parametrize("kind", ["shared", "wide", "small"])
def test_captured_calls_of_every_kind(kind):
    """Each choice of kernels in two graphs, replayed side by side, with lengths that change after the capture."""
    if kind == "shared":
        B, T, Hq, H, ps, shared = 20, 1, 8, 2, 32, 640
        lens = [shared + 5 * b + 1 for b in range(B)]
    elif kind == "wide":
        B, T, Hq, H, ps, shared, lens = 3, 10, 16, 4, 64, 0, [500, 2000, 64]
    else:
        B, T, Hq, H, ps, shared, lens = 2, 1, 8, 2, 64, 0, [900, 1500]
    cache, table, n, q = build(torch.float8_e4m3fn, torch.bfloat16, B, T, Hq, H, 128, ps, lens, shared=shared)
    if kind == "wide":
        table = widen(table, Hq, H, T, ps)
    cache.attend(table, n, q, shared_len=shared)
    q2, n1, n2, side = torch.randn_like(q), n.clone(), n.clone(), torch.cuda.Stream()
    graphs, outs = [], []
    for nn, qq in ((n1, q), (n2, q2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(cache.attend(table, nn, qq, shared_len=shared))
        graphs.append(g)
    n1.copy_(n.flip(0).clamp(max=max(lens)))
    n2[B // 2] = 0
    torch.cuda.synchronize()
    for _ in range(5):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], cache.attend(table, n1, q, shared_len=shared))
    assert torch.equal(outs[1], cache.attend(table, n2, q2, shared_len=shared))


@gpu
def test_output_in_place_of_the_queries():
    for B, T, Hq, H, lens, shared in ((2, 1, 8, 2, [900, 1500], 0), (1, 1, 8, 2, [40000], 0), (20, 1, 8, 2, [700] * 20, 640)):
        cache, table, n, q = build(torch.bfloat16, torch.bfloat16, B, T, Hq, H, 64, 64, lens, shared=shared)
        want = cache.attend(table, n, q, shared_len=shared)
        assert cache.attend(table, n, q, shared_len=shared, out=q) is q
        assert torch.equal(q, want)


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_a_prompt_then_steps_then_tokens(fmt):
    """The operators as a decode loop runs them: a prompt written and attended to in chunks, then steps whose queries
    come from what the cache gave back, tokens drawn from their outputs; every step against 64 bits."""
    from moe_decode_megakernel_02_gb300 import sampling
    B, Hq, H, D, ps, V = 3, 8, 2, 64, 16, 512
    g = torch.Generator(device="cuda").manual_seed(11)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    cache = make_cache(fmt, B * 8, H, ps, D, fill=False)
    table = torch.randperm(B * 8, generator=g, device="cuda").to(torch.int32).view(B, 8)
    head, prompt = rand(Hq * D, V), ints(50, 33, 1)
    at = ints(0, 0, 0)
    for t0 in range(0, 50, 20):  # chunks of 20 tokens; sequences end in different ones
        T = min(20, 50 - t0)
        counts = (prompt - t0).clamp(0, T).to(torch.int32)
        x, y = rand(B, T, H, D).bfloat16(), rand(B, T, H, D).bfloat16()
        cache.write(table, at, x, y, counts=counts)
        at = at + counts
        q = rand(B, T, Hq, D).bfloat16()
        out, lse = cache.attend(table, at, q, return_lse=True)
        check(cache, table, at, q, out, lse, 1 / math.sqrt(D))
    assert at.tolist() == prompt.tolist()
    tokens = torch.zeros(B, dtype=torch.int32, device="cuda")
    for _ in range(4):
        k, v = (torch.zeros((B, 1, H, D), dtype=torch.float32, device="cuda") for _ in range(2))
        cache.read(table, at - 1, k, v)
        x = k + 0.01 * tokens.view(B, 1, 1, 1)
        cache.write(table, at, x, v)
        at = at + 1
        q = x.repeat_interleave(Hq // H, 2).bfloat16()
        out, lse = cache.attend(table, at, q, return_lse=True)
        check(cache, table, at, q, out, lse, 1 / math.sqrt(D))
        logits = out.view(B, Hq * D).float() @ head
        tokens = sampling.sample(logits, torch.rand(B, generator=g, device="cuda"), top_k=ints(1, 20, 0),
                                 temperature=torch.full((B,), 0.7, device="cuda"))
        assert int(tokens[0]) == int(logits[0].argmax()) and bool(((tokens >= 0) & (tokens < V)).all())
        top = logits[1].sort(descending=True).indices[:20]
        assert int(tokens[1]) in top.tolist()


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("ps", [1, 4, 8, 128, 1024])
def test_page_sizes_of_shared_and_wide_calls(fmt, ps):
    """Pages smaller and larger than a tile, and ones too small for the tensor maps."""
    B, Hq, H, D = 5, 16, 2, 128
    shared = max(ps, 192 // ps * ps)
    lens = [shared + 40 * b + 1 for b in range(B)]
    cache, table, n, q = build(fmt, torch.bfloat16, B, 1, Hq, H, D, ps, lens, shared=shared)
    out, lse = cache.attend(table, n, q, shared_len=shared, return_lse=True)
    check(cache, table, n, q, out, lse, 1 / math.sqrt(D))
    T = 5  # 40 rows
    cache, table, n, q = build(fmt, torch.bfloat16, B, T, Hq, H, D, ps, [50, 700, 5, 64, 1100])
    table = widen(table, Hq, H, T, ps)
    out, lse = cache.attend(table, n, q, return_lse=True)
    check(cache, table, n, q, out, lse, 1 / math.sqrt(D))


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_wide_and_shared_calls_past_32_bit_offsets(fmt):
    """Pages whose bytes lie more than 2^32 after the cache's first."""
    H, D, ps = 2, 128, 64
    row = H * ps * D * (2 if fmt == torch.bfloat16 else 1)
    n_pages = (1 << 32) // row + 40
    k, v = (torch.zeros((n_pages, H, ps, D), dtype=torch.int8 if fmt == torch.float8_e4m3fn else fmt, device="cuda")
            for _ in range(2))
    ks, vs = (None, None) if fmt == torch.bfloat16 else (torch.ones((n_pages, H, ps), device="cuda") for _ in range(2))
    cache = pages.Pages(k.view(fmt), v.view(fmt), ks, vs)
    T, Hq, first = 5, 16, n_pages - 20
    table = torch.arange(first, first + 16, dtype=torch.int32, device="cuda").view(1, 16)
    x, y = (torch.randn((1, 16 * ps, H, D), device="cuda").bfloat16() for _ in range(2))
    cache.write(table, ints(0), x, y)
    small = pages.Pages(*(c[first:].contiguous() for c in (cache.k, cache.v)),
                        *(c if c is None else c[first:].contiguous() for c in (ks, vs)))
    q = torch.randn((1, T, Hq, D), device="cuda").bfloat16()
    for t, kw in ((widen(table, Hq, H, T, ps), {}), (table, dict(shared_len=512))):
        t0 = torch.where(t < 0, t, t - first)
        a = cache.attend(t, ints(1000), q, **kw)
        assert torch.equal(a, small.attend(t0, ints(1000), q, **kw)) and bool((a != 0).any())
