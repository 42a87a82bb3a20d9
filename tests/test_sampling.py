"""Sampling from logits: refusals (CPU), mk_sample against its definition in 64 bits, and the sampled decode loop.

The kernel's weights are 32-bit exponentials (at most 2 steps of 2^-23 off, after an exponent rounded to 32 bits);
sums are exact to 2^-42. Against weights of 64 bits a running sum of the kept tokens is therefore off by at most
delta = 2^-22 + 2^-24 (max exponent + 1) of the total, so the token must be one whose span of the running sum
reaches within delta of u. Where a filter's border lies within delta of p (or a weight within delta of min_p) both
sides of it are allowed. Rows made of a few exactly equal logits have exact answers and are compared as such.
"""
import ctypes
import math

import pytest
import torch

import moe_decode_megakernel_02_gb300 as mk
from moe_decode_megakernel_02_gb300 import sampling

gpu = pytest.mark.gpu


def _struct(**over):
    a = dict(logits=4096, row_stride=100, u=4096, temperature=None, top_k=None, top_p=None, min_p=None, tokens=4096,
             probs=None, kept=None, rows=1, vocab=100, dtype=mk.DT_F32, reserved=0)
    a.update(over)
    return mk.SamplingStruct(**a)


@pytest.mark.parametrize("over,code", [
    (dict(logits=None), mk.ERR_INVALID_ARG), (dict(u=None), mk.ERR_INVALID_ARG), (dict(tokens=None), mk.ERR_INVALID_ARG),
    (dict(rows=-1), mk.ERR_INVALID_ARG), (dict(vocab=0), mk.ERR_INVALID_ARG), (dict(dtype=3), mk.ERR_INVALID_ARG),
    (dict(logits=4097), mk.ERR_INVALID_ARG), (dict(vocab=360449), mk.ERR_UNSUPPORTED),
    (dict(rows=(1 << 31) - 1), mk.ERR_UNSUPPORTED),
])
def test_bad_arguments_are_refused(over, code):
    assert mk.lib().mk_sample(ctypes.byref(_struct(**over)), None) == code
    assert mk.lib().mk_last_error()
    assert mk.lib().mk_sample(None, None) == mk.ERR_INVALID_ARG


def test_no_rows_is_nothing_to_do():
    assert mk.lib().mk_sample(ctypes.byref(_struct(rows=0, logits=None, tokens=None, u=None)), None) == mk.OK


def _allowed(x, u, T, k, p, least):
    """(tokens that 64-bit weights allow, least and largest count kept) of one row."""
    x = x.double()
    if bool((x == math.inf).any()) or bool(torch.isnan(x).any()) or bool((x == -math.inf).all()):
        return {-1}, 0, 0
    order = torch.sort(x, descending=True, stable=True).indices
    if not T > 0:
        return {int(order[0])}, 1, 1
    z = (x - x.max()) / T
    w = z.exp()
    delta = 2.0 ** -22 + 2.0 ** -24 * (float(z[z > -200].abs().max()) + 1)
    order = order[x[order] > -math.inf]
    if k > 0:
        order = order[:k]
    ws = w[order]
    before = (ws.cumsum(0) - ws) / ws.sum()
    spans = []
    for sign in (-1, 1):
        keep = torch.ones_like(ws, dtype=torch.bool)
        if p < 1:
            keep &= before < p + sign * delta
        keep &= ws >= least * (1 - sign * 4 * delta)
        keep[0] = True
        spans.append(keep)
    allowed = set()
    for keep in spans:
        ids = order[keep].sort().values
        c = w[ids].cumsum(0) / w[ids].sum()
        lo, hi = c - w[ids] / w[ids].sum(), c
        # a border token more or less moves every span by at most its own share
        shift = float((ws[spans[1] & ~spans[0]]).sum() / ws[spans[0]].sum())
        uu = min(max(u, 0.0), 1 - 2.0 ** -24)
        ok = (lo <= uu + delta + shift) & (hi >= uu - delta - shift)
        allowed |= set(ids[ok].tolist())
    return allowed, int(spans[0].sum()), int(spans[1].sum())


def check(logits, u, T, k, p, least):
    tok, prob, kept = sampling.sample(logits, u, temperature=T, top_k=k, top_p=p, min_p=least, return_details=True)
    tok2 = sampling.sample(logits, u, temperature=T, top_k=k, top_p=p, min_p=least)
    assert torch.equal(tok, tok2)
    one = lambda v, r, d: d if v is None else float(v[r])  # noqa: E731
    for r in range(logits.shape[0]):
        allowed, lo, hi = _allowed(logits[r].float(), float(u[r]), one(T, r, 1.0), int(one(k, r, 0)), one(p, r, 1.0),
                                   one(least, r, 0.0))
        assert int(tok[r]) in allowed, (r, int(tok[r]), sorted(allowed)[:5])
        assert lo <= int(kept[r]) <= hi, (r, int(kept[r]), lo, hi)
    assert bool(((prob > 0) == (tok >= 0)).all()) and bool((prob <= 1).all())
    return tok, prob, kept


def settings(R, g):
    def pick(values, dtype):
        return torch.tensor(values, device="cuda", dtype=dtype)[torch.randint(0, len(values), (R,), generator=g,
                                                                              device="cuda")]
    return (pick([1.0, 0.7, 1.5, 0.0, 0.05, 50.0], torch.float32), pick([0, 1, 2, 20, 1000, -3, 1 << 30], torch.int32),
            pick([1.0, 0.9, 0.5, 0.0, 0.99, 2.0], torch.float32), pick([0.0, 0.05, 0.5, 1.0], torch.float32))


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("R,V", [(1, 1), (3, 2), (5, 31), (40, 1024), (9, 2049), (7, 4097), (4, 16385), (3, 64000),
                                 (2, 151936)])
def test_tokens_match_the_definition(dtype, R, V):
    g = torch.Generator(device="cuda").manual_seed(V)
    x = (torch.randn((R, V), generator=g, device="cuda") * 3).to(dtype)
    u = torch.rand((R,), generator=g, device="cuda")
    u[0] = 0.0
    check(x, u, None, None, None, None)
    check(x, u, *settings(R, g))


@gpu
def test_the_largest_vocabulary():
    V = 360448
    x = torch.randn((1, V), device="cuda")
    check(x, torch.tensor([0.73], device="cuda"), torch.tensor([1.2], device="cuda"), ints(50000),
          torch.tensor([0.93], device="cuda"), None)
    x[0, V - 1] = 90.0
    assert int(sampling.sample(x, torch.tensor([0.5], device="cuda"))) == V - 1


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def floats(*v):
    return torch.tensor(v, dtype=torch.float32, device="cuda")


@gpu
@pytest.mark.parametrize("V", [8, 5000])
def test_ties_go_to_the_lowest_index(V):
    """Equal logits: every border falls among ties, and all sums are whole numbers of one weight."""
    x = torch.zeros((6, V), device="cuda")
    x[4, 3] = -0.0  # equal to 0
    h = V // 2
    tok, prob, kept = sampling.sample(
        x, floats(0.0, 0.999999, 0.5, 0.999999, 0.999999, 0.25), temperature=floats(1, 1, 1, 2, 1, 0),
        top_k=ints(0, h, 0, h, 4, 5), top_p=floats(1, 1, 0.5, 0.5, 1, 1), return_details=True)
    assert kept.tolist() == [V, h, h, h // 2, 4, 1]
    assert tok.tolist() == [0, h - 1, h // 2, h // 2 - 1, 3, 0]
    assert torch.equal(prob, 1 / kept.float())
    # the ties of top-k's border count for top-p with those that are kept
    y = torch.full((1, V), -1.0, device="cuda")
    y[0, -1] = 2.0
    tok, prob, kept = sampling.sample(y, floats(0.999999), top_k=ints(4), top_p=floats(0.9999), return_details=True)
    assert kept.tolist() == [4] and tok.tolist() == [V - 1]
    tok, _, kept = sampling.sample(y, floats(0.0), top_k=ints(4), top_p=floats(0.9999), return_details=True)
    assert tok.tolist() == [0]


@gpu
def test_masked_tokens_and_rows_without_a_distribution():
    V = 3000
    x = torch.randn((7, V), device="cuda")
    x[0] = -math.inf
    x[1, 5] = math.nan
    x[2, 6] = math.inf
    x[3] = -math.inf
    x[3, 17] = -3e38
    x[4, ::2] = -math.inf
    x[5] = torch.finfo(torch.float32).min
    x[6] = -math.inf
    x[6, :3] = floats(3e38, -3e38, 3e38)
    u = floats(.5, .5, .5, .5, .999, .5, .9)
    for kw in (dict(), dict(top_k=ints(*[2000] * 7)), dict(top_p=floats(*[0.999] * 7)),
               dict(temperature=floats(*[1e-30] * 7)), dict(temperature=floats(*[1e30] * 7)),
               dict(temperature=floats(*[0.0] * 7)), dict(temperature=floats(*[math.inf] * 7))):
        tok, prob, kept = sampling.sample(x, u, return_details=True, **kw)
        assert tok[:4].tolist() == [-1, -1, -1, 17] and kept[:4].tolist() == [0, 0, 0, 1]
        assert prob[:4].tolist() == [0, 0, 0, 1]
        assert int(tok[4]) % 2 == 1 and 0 <= int(tok[5]) < V and int(tok[6]) in (0, 1, 2)
        assert int(kept[4]) <= V // 2
    tok, _, kept = sampling.sample(x, u, return_details=True)
    assert int(kept[4]) == V // 2 and int(kept[5]) == V and int(tok[5]) == V // 2 and int(kept[6]) == 3
    assert int(tok[6]) == 2


@gpu
def test_odd_settings():
    x = torch.tensor([[1.0, 3.0, 2.0, 3.0]], device="cuda").repeat(8, 1)
    nan = math.nan
    tok, _, kept = sampling.sample(
        x, floats(0.999999, 0.999999, -1.0, 2.0, nan, 0.6, 0.6, 0.6), temperature=floats(1, 1, 1, 1, 1, nan, -2, 1),
        top_k=ints(0, 0, 0, 0, 0, 0, 0, 3), top_p=floats(-1, nan, 1, 1, 1, 1, 1, 1),
        min_p=floats(0, 0, 0, 0, 0, 0, 0, 7), return_details=True)
    # p <= 0 and min_p > 1 keep the first rank; a NaN p is no filter; u is held in [0, 1); T NaN or <= 0 is greedy
    assert kept.tolist() == [1, 4, 4, 4, 4, 1, 1, 1]
    assert tok.tolist() == [1, 3, 0, 3, 0, 1, 1, 1]


@gpu
def test_strides_streams_and_graphs():
    R, V = 6, 5000
    wide = torch.randn((R, V + 7), device="cuda")
    x = wide[:, 3:3 + V]
    u = torch.rand(R, device="cuda")
    p = floats(*[0.9] * R)
    want = sampling.sample(x.contiguous(), u, top_p=p)
    assert torch.equal(sampling.sample(x, u, top_p=p), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sampling.sample(x, u, top_p=p, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty(R, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sampling.sample(x, u, top_p=p, out=out)
    u.copy_(torch.rand(R, device="cuda"))
    g.replay()
    assert torch.equal(out, sampling.sample(x, u, top_p=p))


@gpu
def test_frequencies_follow_the_weights():
    """20,000 rows of one distribution: each token's count within 6 standard deviations."""
    R, V = 20000, 16
    x = torch.linspace(-2, 2, V, device="cuda").repeat(R, 1)
    u = (torch.arange(R, device="cuda", dtype=torch.float32) + 0.5) / R
    tok = sampling.sample(x, u).long()
    want = torch.softmax(x[0].double(), 0) * R
    # u runs over an even grid: every count is within 2 of its share
    assert bool(((torch.bincount(tok, minlength=V) - want).abs() <= 2).all())


@gpu
def test_binding_refuses_what_does_not_fit():
    x, u = torch.randn((2, 50), device="cuda"), torch.rand(2, device="cuda")
    for args, kw in (((x.double(), u), {}), ((x.cpu(), u.cpu()), {}), ((x[0], u), {}), ((x.t(), u), {}), ((x, None), {}),
                     ((x, u.double()), {}), ((x, u[:1]), {}), ((x, u), dict(top_k=u)), ((x, u), dict(out=u)),
                     ((x, u), dict(temperature=u.cpu()))):
        with pytest.raises(ValueError):
            sampling.sample(*args, **kw)
    assert sampling.sample(x[:0], u[:0]).shape == (0,)


@gpu
def test_sampled_decode_loop():
    """Temperature 0 reproduces greedy steps; sampled tokens follow from the step's logits and the same u."""
    from moe_decode_megakernel_02_gb300 import workload
    from synth import configs
    cfg = configs.TINY
    ctx, B, steps = cfg["ctx"], 2, 5
    model = workload.load_synthetic(cfg, max_batch=B, max_tokens_per_seq=1, max_ctx=ctx + 16)
    first = workload.tokens(cfg, 0, B, 1)[:, 0]

    def fresh():
        kv = mk.KVCache(model, B, ctx + 16)
        workload.prefill(kv, cfg, ctx)
        return kv

    greedy = sampling.SampledLoop(model, fresh(), first, [ctx] * B, cfg["vocab"], temperature=0.0)
    kv, tok = fresh(), torch.from_numpy(first.copy()).cuda().view(B, 1)
    logits = torch.empty((B, cfg["vocab"]), device="cuda")
    for i in range(steps):
        greedy.step()
        model.decode_step(kv, tok, ints(*[ctx + i] * B), logits)
        tok = logits.argmax(-1).to(torch.int32).view(B, 1)
        assert torch.equal(tok[:, 0], greedy.emitted[-1])
    assert len(greedy.tokens()) == B and len(greedy.tokens()[0]) == steps
    g = torch.Generator(device="cuda").manual_seed(5)
    loop = sampling.SampledLoop(model, fresh(), first, [ctx] * B, cfg["vocab"], temperature=[1.0, 0.8], top_k=40,
                                top_p=0.95, generator=g)
    for i in range(steps):
        drawn = loop.step()
        assert torch.equal(drawn, sampling.sample(loop.logits, loop.u, **loop.settings))
        assert bool(((drawn >= 0) & (drawn < cfg["vocab"])).all())
    assert loop.tokens()[0] == [int(t[0]) for t in loop.emitted]
    with pytest.raises(ValueError):
        sampling.SampledLoop(model, fresh(), first, [ctx] * B, cfg["vocab"], temperature=[1.0] * 3)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_borders_that_fit_no_list(dtype):
    """Long runs of equal and nearly equal logits, large k, and one thread's share of the row holding all that counts."""
    V = 40000
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros((8, V), device="cuda")
    x[1] = torch.randn(V, generator=g, device="cuda") * 1e-4        # all in one bin
    x[2] = torch.randn(V, generator=g, device="cuda")
    x[3] = torch.randint(0, 3, (V,), generator=g, device="cuda").float()
    x[4, 20000:] = -math.inf
    x[5] = torch.linspace(5, -5, V, device="cuda")                  # sorted: the largest lie side by side
    x[6, ::4096] = 3.0                                              # the largest at one stride
    x[7] = -torch.arange(V, device="cuda").float() / 7
    x = x.to(dtype)
    u = torch.rand(8, generator=g, device="cuda")
    for k in (0, 3, 1500, 9999, 30000):
        for p in (1.0, 0.5, 0.97):
            check(x, u, floats(*[0.9] * 8), ints(*[k] * 8), floats(*[p] * 8), floats(0, 0, 0, 0.2, 0, 0, 0.01, 0.001))
    # equal logits: exact counts and tokens
    tok, _, kept = sampling.sample(x[:1].repeat(4, 1), floats(0, 0.5, 0.999999, 0.999999), top_k=ints(0, 9000, 9000, 9000),
                                   top_p=floats(0.5, 1.0, 0.5, 1.0), return_details=True)
    assert kept.tolist() == [20000, 9000, 4500, 9000] and tok.tolist() == [0, 4500, 4499, 8999]


@pytest.mark.parametrize("name", ["u", "temperature", "top_k", "top_p", "min_p", "tokens", "probs", "kept"])
def test_unaligned_arrays_are_refused(name):
    assert mk.lib().mk_sample(ctypes.byref(_struct(**{name: 4098})), None) == mk.ERR_INVALID_ARG


@gpu
def test_two_calls_at_once_and_replayed():
    """Every kind of filter in graphs replayed side by side, on rows that change after the capture."""
    R, V = 12, 30000
    x = torch.randn((R, V), device="cuda") * 2
    y, u = torch.randn_like(x), torch.rand(R, device="cuda")
    kinds = (dict(), dict(top_k=ints(*[30] * R)), dict(top_p=floats(*[0.9] * R)),
             dict(top_k=ints(*[900] * R), top_p=floats(*[0.95] * R), min_p=floats(*[0.001] * R)),
             dict(temperature=floats(*[0.0] * R)))
    graphs, outs = [], []
    for src in (x, y):
        for kw in kinds:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs.append(sampling.sample(src, u, return_details=True, **kw))
            graphs.append(g)
    x.copy_(torch.randn_like(x))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(len(kinds)):
            graphs[i].replay()
            with torch.cuda.stream(side):
                graphs[len(kinds) + i].replay()
    torch.cuda.synchronize()
    want = [sampling.sample(src, u, return_details=True, **kw) for src in (x, y) for kw in kinds]
    for got, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(got, w))


@gpu
@pytest.mark.parametrize("R", [330, 2048, 2049])
def test_many_rows_give_what_few_do(R):
    """More rows than run at once are taken in another order: every row's result is that of a call of its own size."""
    V = 8200
    g = torch.Generator(device="cuda").manual_seed(R)
    x = torch.randn((R, V), generator=g, device="cuda") * 3
    u = torch.rand((R,), generator=g, device="cuda")
    T, k, p, least = settings(R, g)
    cases = ((T, k, p, least), (None, None, p, None), (None, None, torch.ones_like(p), None))
    for T, k, p, least in cases:
        got = sampling.sample(x, u, temperature=T, top_k=k, top_p=p, min_p=least, return_details=True)
        for r in range(0, R, 100):
            cut = lambda v: None if v is None else v[r:r + 100]  # noqa: E731
            want = sampling.sample(x[r:r + 100], cut(u), temperature=cut(T), top_k=cut(k), top_p=cut(p), min_p=cut(least),
                                   return_details=True)
            assert all(torch.equal(a[r:r + 100], b) for a, b in zip(got, want))
