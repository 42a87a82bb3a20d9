"""Causal attention of prompts over expanded keys and values, against the definition in 64 bits.

Tolerance, as in test_latent with heads of 192: scores lose (192 + 8) 2^-23 of sum |q k| scale, weights twice that,
and eps/2 for their rounding to the values' type (fp16: at least 2^-25 of the largest); 32-bit sums 2^-18; the result is
rounded once.
"""
import ctypes
import math

import pytest
import torch

import moe_decode_megakernel_02_gb300 as mk
from moe_decode_megakernel_02_gb300 import latent

gpu = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def starts(sizes, first=0):
    at = [first]
    for n in sizes:
        at.append(at[-1] + n)
    return ints(*at)


def make(dtype, nq, nk, H, seed=0, spare=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    N, M = sum(nq) + spare, sum(nk) + spare

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    kv = normal(M, H, 256)
    return normal(N, H, 192), kv[..., :128], normal(M, 64), kv[..., 128:]


def check(q, k, r, v, q_at, k_at, scale, out, lse):
    half = torch.finfo(q.dtype).eps / 2
    q_at, k_at = q_at.tolist(), k_at.tolist()
    for b in range(len(q_at) - 1):
        n, m = q_at[b + 1] - q_at[b], k_at[b + 1] - k_at[b]
        if n == 0:
            continue
        rows, keys = slice(q_at[b], q_at[b + 1]), slice(k_at[b], k_at[b + 1])
        qq, kk, vv = q[rows].double(), k[keys].double(), v[keys].double()
        kk = torch.cat([kk, r[keys].double()[:, None].expand(-1, q.shape[1], -1)], -1)
        x = torch.einsum("nhd,mhd->hnm", qq, kk) * scale
        hidden = torch.arange(m, device="cuda") > (m - n + torch.arange(n, device="cuda"))[:, None]
        size = (torch.einsum("nhd,mhd->hnm", qq.abs(), kk.abs()) * abs(scale)).masked_fill(hidden, 0)
        e = (200 * 2.0 ** -23 * size.amax(-1)).T if m else torch.zeros(n, q.shape[1], device="cuda")  # [n, H]
        x = x.masked_fill(hidden, -math.inf)
        want_lse = torch.logsumexp(x, -1).T if m else torch.full((n, q.shape[1]), -math.inf, device="cuda")
        none = want_lse == -math.inf
        w = torch.softmax(x, -1).nan_to_num(0)
        want = torch.einsum("hnm,mhd->nhd", w, vv)
        bound = torch.einsum("hnm,mhd->nhd", w, vv.abs()) * (2 * e + half + 2.0 ** -18)[..., None] + want.abs() * half
        if q.dtype == torch.float16:
            bound = bound + 2.0 ** -25 * (1 + torch.einsum("nm,mhd->nhd", (~hidden).double(), vv.abs()))
        err = (out[rows].double() - want).abs()
        assert (err <= bound).all(), (b, (err - bound).max().item(), (err > bound).nonzero()[0].tolist())
        assert (out[rows][none] == 0).all()
        if lse is not None:
            got = lse[rows].double()
            assert torch.equal(got == -math.inf, none)
            assert ((got - want_lse).abs()[~none] <= (e + 2.0 ** -18 + want_lse.abs() * 2.0 ** -22)[~none]).all()


# ---------------------------------------------------------------- refusals (CPU)

def _args(**over):
    one = 4096  # aligned, never followed
    a = dict(q_starts=one, k_starts=one, q=one, k=one, k_rope=one, v=one, out=one, lse=None, status=None, q_token=384,
             q_head=192, k_token=256, k_head=128, rope_token=64, v_token=256, v_head=128, out_token=256, out_head=128,
             batch=1, n_tokens=4, n_keys=4, n_heads=2, nope_dim=128, rope_dim=64, v_dim=128, dtype=mk.DT_BF16, scale=0.1,
             reserved=0)
    return mk.PromptAttentionStruct(**{**a, **over})


@pytest.mark.parametrize("over,code", [
    (dict(q_starts=None), mk.ERR_INVALID_ARG), (dict(k_starts=None), mk.ERR_INVALID_ARG),
    (dict(q_starts=4098), mk.ERR_INVALID_ARG), (dict(lse=4098), mk.ERR_INVALID_ARG),
    (dict(status=4097), mk.ERR_INVALID_ARG), (dict(q=None), mk.ERR_INVALID_ARG), (dict(k=None), mk.ERR_INVALID_ARG),
    (dict(k_rope=None), mk.ERR_INVALID_ARG), (dict(v=None), mk.ERR_INVALID_ARG), (dict(out=None), mk.ERR_INVALID_ARG),
    (dict(q=4104), mk.ERR_INVALID_ARG), (dict(v=4104), mk.ERR_INVALID_ARG), (dict(out=4098), mk.ERR_INVALID_ARG),
    (dict(q_token=388), mk.ERR_INVALID_ARG), (dict(k_head=132), mk.ERR_INVALID_ARG),
    (dict(rope_token=-64), mk.ERR_INVALID_ARG), (dict(dtype=mk.DT_F32), mk.ERR_INVALID_ARG),
    (dict(batch=0), mk.ERR_INVALID_ARG), (dict(n_tokens=-1), mk.ERR_INVALID_ARG), (dict(n_keys=-1), mk.ERR_INVALID_ARG),
    (dict(n_heads=0), mk.ERR_INVALID_ARG), (dict(scale=math.nan), mk.ERR_INVALID_ARG),
    (dict(scale=math.inf), mk.ERR_INVALID_ARG), (dict(nope_dim=64), mk.ERR_UNSUPPORTED),
    (dict(rope_dim=32), mk.ERR_UNSUPPORTED), (dict(v_dim=64), mk.ERR_UNSUPPORTED),
    (dict(n_tokens=1 << 30), mk.ERR_UNSUPPORTED), (dict(n_keys=(1 << 30) + 1), mk.ERR_UNSUPPORTED),
    (dict(batch=1 << 21), mk.ERR_UNSUPPORTED), (dict(n_tokens=0), mk.OK),
])
def test_refusals(over, code):
    assert mk.lib().mk_prompt_attend(ctypes.byref(_args(**over)), None) == code
    assert mk.lib().mk_prompt_attend(None, None) == mk.ERR_INVALID_ARG


# ---------------------------------------------------------------- on the GPU

@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("nq,ctx,H", [
    ([1], [0], 1), ([1], [200], 3), ([2], [0], 16), ([64], [0], 2), ([127], [0], 1), ([128], [0], 2), ([129], [0], 5),
    ([255, 1, 256], [0, 0, 0], 2), ([300], [77], 3), ([5, 0, 130, 64], [300, 10, 0, 64], 2), ([1000], [0], 4),
    ([1] * 40, list(range(40)), 2), ([513, 31], [511, 2000], 1), ([700, 3, 90], [0, 1, 129], 16),
])
def test_against_the_definition(dtype, nq, ctx, H):
    nk = [n + c for n, c in zip(nq, ctx)]
    q, k, r, v = make(dtype, nq, nk, H)
    q_at, k_at = starts(nq), starts(nk)
    out, lse = latent.attend_prompt(q, k, r, v, q_at, k_at, 192 ** -0.5, return_lse=True)
    check(q, k, r, v, q_at, k_at, 192 ** -0.5, out, lse)
    assert torch.equal(latent.attend_prompt(q, k, r, v, q_at, k_at, 192 ** -0.5), out)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_queries_that_see_nothing(dtype):
    """More queries than keys: the first ones see none; a sequence without keys at all."""
    nq, nk = [200, 5, 130], [130, 0, 1]
    q, k, r, v = make(dtype, nq, nk, 2)
    q_at, k_at = starts(nq), starts(nk)
    out, lse = latent.attend_prompt(q, k, r, v, q_at, k_at, 0.1, return_lse=True)
    check(q, k, r, v, q_at, k_at, 0.1, out, lse)
    out, lse = latent.attend_prompt(q[:9], k[:0], r[:0], v[:0], ints(0, 9), ints(0, 0), 0.1, return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("junk", [math.nan, math.inf, 65504.0])
def test_keys_behind_a_query_cannot_reach_it(dtype, junk):
    nq, nk = [150, 70], [200, 70]
    q, k, r, v = make(dtype, nq, nk, 2, spare=300)
    q_at, k_at = starts(nq), starts(nk)
    want = latent.attend_prompt(q, k, r, v, q_at, k_at, 0.07)
    for x in (k, r, v):
        x[170:200] = junk   # behind query 119 of the first sequence
        x[230:] = junk      # behind query 29 of the second, and rows of nobody
    got = latent.attend_prompt(q, k, r, v, q_at, k_at, 0.07)
    assert torch.equal(got[:120], want[:120]) and torch.equal(got[150:180], want[150:180])


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_scores_far_apart(dtype):
    nq, nk = [333], [333]
    q, k, r, v = make(dtype, nq, nk, 2)
    q_at, k_at = starts(nq), starts(nk)
    for scale in (3.0, -0.3, 0.0):
        out, lse = latent.attend_prompt(q, k, r, v, q_at, k_at, scale, return_lse=True)
        check(q, k, r, v, q_at, k_at, scale, out, lse)
    j = torch.arange(333, device="cuda", dtype=torch.float32)
    for slope in (0.5, -0.5):  # scores that rise past every tile's, or fall
        q.zero_(), r.zero_()
        q[..., 128], r[:, 0] = 1, (j * slope).to(dtype)
        out, lse = latent.attend_prompt(q, k, r, v, q_at, k_at, 1.0, return_lse=True)
        check(q, k, r, v, q_at, k_at, 1.0, out, lse)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_rows_of_nobody(dtype):
    """Heads before tokens, a rope part inside a wider row, an output inside another; rows before the first and behind the
    last sequence stay."""
    H, N = 3, 260
    q = torch.randn((H, N, 200), device="cuda").to(dtype).transpose(0, 1)[..., 8:]
    k = torch.randn((H, N, 128), device="cuda").to(dtype).transpose(0, 1)
    v = torch.randn((N, H, 136), device="cuda").to(dtype)[..., :128]
    r = torch.randn((N, 576), device="cuda").to(dtype)[:, 512:]
    q_at, k_at = ints(10, 150, 240), ints(3, 143, 260)
    room = torch.full((N, H, 144), 7.0, device="cuda").to(dtype)
    out = room[..., 8:136]
    got, lse = latent.attend_prompt(q, k, r, v, q_at, k_at, 0.07, out=out, return_lse=True)
    assert got is out
    check(q, k, r, v, q_at, k_at, 0.07, out, lse)
    assert (out[:10] == 7).all() and (out[240:] == 7).all()
    out[10:240] = 7.0
    assert (room == 7.0).all()


@gpu
@pytest.mark.parametrize("q_at,k_at", [([0, 60, 40, 100], [0, 60, 80, 100]), ([0, 20, 40, 200], [0, 20, 40, 60]),
                                       ([0, 20, 40, 60], [0, 20, 40, 101]), ([0, 20, 40, 60], [0, 50, 20, 60]),
                                       ([-5, 20, 40, 60], [0, 20, 40, 60]), ([0, 20, 40, 60], [-9, 20, 40, 60])])
def test_bounds_out_of_range_skip_their_sequence(q_at, k_at):
    q, k, r, v = make(torch.bfloat16, [100], [100], 2)
    status = ints(0)
    out = torch.full((100, 2, 128), 7.0, device="cuda").bfloat16()
    lse = latent.attend_prompt(q, k, r, v, ints(*q_at), ints(*k_at), 0.1, out=out, return_lse=True, status=status)[1]
    assert status.item() == mk.ERR_INVALID_ARG
    for b in range(3):
        a, e, c, d = q_at[b], q_at[b + 1], k_at[b], k_at[b + 1]
        good = 0 <= a <= e <= 100 and 0 <= c <= d <= 100
        # (bounds that descend: another sequence's rows may be among this one's)
        if good and all(x <= a or x >= e for i, x in enumerate(q_at) if i not in (b, b + 1)):
            check(q, k, r, v, ints(a, e), ints(c, d), 0.1, out, lse)


@gpu
def test_captured_and_on_a_stream():
    nq, nk = [100, 31], [164, 31]
    q, k, r, v = make(torch.bfloat16, nq, nk, 4)
    q_at, k_at = starts(nq), starts(nk)
    graph = torch.cuda.CUDAGraph()
    latent.attend_prompt(q, k, r, v, q_at, k_at, 0.07)
    with torch.cuda.graph(graph):
        out = latent.attend_prompt(q, k, r, v, q_at, k_at, 0.07)
    q_at.copy_(ints(0, 30, 131))
    k_at.copy_(ints(0, 30, 195))
    v.normal_()
    graph.replay()
    assert torch.equal(out, latent.attend_prompt(q, k, r, v, q_at, k_at, 0.07))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = latent.attend_prompt(q, k, r, v, q_at, k_at, 0.07, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, out)


@gpu
def test_chunks_equal_the_whole():
    """A prompt taken in chunks behind their contexts, as a server does it, is the prompt taken at once."""
    n = 700
    q, k, r, v = make(torch.bfloat16, [n], [n], 2)
    whole = latent.attend_prompt(q, k, r, v, ints(0, n), ints(0, n), 0.07)
    at = 0
    for size in (1, 255, 64, 380):
        part = latent.attend_prompt(q[at:at + size], k[:at + size], r[:at + size], v[:at + size], ints(0, size),
                                    ints(0, at + size), 0.07)
        check(q[at:at + size], k, r, v, ints(0, size), ints(0, at + size), 0.07, part, None)
        assert (part.float() - whole[at:at + size].float()).abs().max() <= 2 * 2.0 ** -7 * whole.float().abs().max()
        at += size


@gpu
def test_the_bindings_refusals():
    q, k, r, v = make(torch.bfloat16, [10], [10], 2)
    at = ints(0, 10)
    good = dict(q=q, k=k, k_rope=r, v=v, q_starts=at, k_starts=at, scale=0.1)
    for over in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[0]), dict(k=k.half()), dict(k=k[:, :1]), dict(k=k[:5]),
                 dict(k_rope=r[:5]), dict(k_rope=r[:, :32]), dict(v=v[:5]), dict(v=v.float()), dict(q_starts=None),
                 dict(q_starts=at.long()), dict(q_starts=at[:1]), dict(k_starts=ints(0, 5, 10)), dict(out=q),
                 dict(out=torch.empty((10, 2, 128), device="cuda")), dict(scale="x"), dict(status=at),
                 dict(out=torch.empty((1, 2, 128), device="cuda", dtype=torch.bfloat16).expand(10, 2, 128)),
                 dict(q=q.transpose(1, 2))):
        with pytest.raises(ValueError):
            latent.attend_prompt(**{**good, **over})
    with pytest.raises(mk.MKError):
        latent.attend_prompt(**{**good, "scale": math.nan})
    with pytest.raises(mk.MKError):  # heads of another size
        latent.attend_prompt(q[..., :128], k[..., :64], r, v, at, at, 0.1)
    assert latent.attend_prompt(q[:0], k, r, v, ints(0, 0), at, 0.1).shape == (0, 2, 128)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("nq,ctx,H", [
    ([1], [3000], 1), ([1], [20000], 2), ([200], [9000], 3), ([64, 1], [5000, 1000], 1), ([300], [2000], 5), ([257], [1024], 1),
    ([5, 5, 5], [2100, 0, 4000], 2), ([130], [16000], 1), ([1000], [0], 3),
])
def test_few_queries_behind_long_contexts(dtype, nq, ctx, H):
    """Blocks whose keys several CTAs share, parts without a tile of a block among them."""
    nk = [n + c for n, c in zip(nq, ctx)]
    q, k, r, v = make(dtype, nq, nk, H)
    q_at, k_at = starts(nq), starts(nk)
    out, lse = latent.attend_prompt(q, k, r, v, q_at, k_at, 192 ** -0.5, return_lse=True)
    check(q, k, r, v, q_at, k_at, 192 ** -0.5, out, lse)
    if len(nq) == 1 and nq[0] > 1:  # the newest key is the last query's alone
        k[-1] = r[-1] = v[-1] = math.nan
        again = latent.attend_prompt(q, k, r, v, q_at, k_at, 192 ** -0.5)
        assert torch.equal(again[:-1], out[:-1]) and again[-1].isnan().all()
