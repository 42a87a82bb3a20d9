"""Log probabilities, entropies and alternatives, against the definition in 64 bits.

Tolerance. z = (x - max) / T is off by 2^-22 of itself, e^z by 2^-22 + 2^-22 |z| of itself; a sum of V terms in 32 bits,
at least 256 of them added in turn by different threads, by less than (V / 256 + 32) 2^-24 of it. A log probability is z
less a logarithm whose argument is off by these (the weights of large |z| are small: sum p |z| is the entropy's size),
an entropy the logarithm plus a quotient of two such sums.
"""
import ctypes
import math
import types

import pytest
import torch

import moe_decode_megakernel_02_gb300 as mk
from moe_decode_megakernel_02_gb300 import sampling

gpu = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def expected(x, T):
    x = x.double()
    z = x if T is None else x / T.double()[:, None]
    logp = torch.log_softmax(z, -1)
    p = logp.exp()
    h = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(-1)
    spread = torch.where(p > 0, p * (z - z.amax(-1, keepdim=True)).abs(), torch.zeros_like(p)).sum(-1)
    return logp, h, spread


def check(x, tokens, top, T=None):
    R, V = x.shape
    got, entropy, ids, best = sampling.logprobs(x, tokens, top=top, temperature=T)
    logp, h, spread = expected(x, T)
    base = (V / 256 + 32) * 2.0 ** -24 + 2.0 ** -21 * (1 + spread)

    def close(a, b, tol):
        far = (a.double() - b).abs() <= tol
        assert (far | (a.double() == b)).all(), (a.double() - b).abs().max()

    if tokens is not None:
        want = logp.gather(1, tokens.long().view(R, -1)).view(tokens.shape)
        tol = base.view(-1, *[1] * (tokens.dim() - 1)) + want.abs() * 2.0 ** -21
        close(got, want, tol)
    else:
        assert got is None
    close(entropy, h, base * (1 + spread) * 2)
    order = x.float().sort(dim=-1, descending=True, stable=True).indices[:, :top]
    assert ids.dtype == torch.int32 and torch.equal(ids.long(), order)
    want = logp.gather(1, order)
    close(best, want, base[:, None] + want.abs() * 2.0 ** -21)


# ---------------------------------------------------------------- without a GPU

def _args(**over):
    one = 4096
    a = dict(logits=one, row_stride=100, temperature=None, tokens=one, logprobs=one, entropy=one, top_ids=one,
             top_logprobs=one, rows=2, vocab=100, dtype=mk.DT_F32, given=1, top=5, reserved=0)
    return mk.LogprobStruct(**{**a, **over})


@pytest.mark.parametrize("over,code", [
    (dict(logits=None), mk.ERR_INVALID_ARG), (dict(logits=4098), mk.ERR_INVALID_ARG), (dict(dtype=5), mk.ERR_INVALID_ARG),
    (dict(rows=-1), mk.ERR_INVALID_ARG), (dict(vocab=0), mk.ERR_INVALID_ARG), (dict(given=-1), mk.ERR_INVALID_ARG),
    (dict(top=-1), mk.ERR_INVALID_ARG), (dict(top=101), mk.ERR_INVALID_ARG), (dict(top=65), mk.ERR_UNSUPPORTED),
    (dict(vocab=(1 << 30) + 1), mk.ERR_UNSUPPORTED),
    (dict(tokens=None), mk.ERR_INVALID_ARG), (dict(logprobs=None), mk.ERR_INVALID_ARG),
    (dict(top_ids=None), mk.ERR_INVALID_ARG), (dict(top_logprobs=None), mk.ERR_INVALID_ARG),
    (dict(tokens=4098), mk.ERR_INVALID_ARG), (dict(temperature=4097), mk.ERR_INVALID_ARG),
    (dict(entropy=4097), mk.ERR_INVALID_ARG), (dict(row_stride=-100), mk.ERR_INVALID_ARG), (dict(rows=0), mk.OK),
])
def test_refusals(over, code):
    assert mk.lib().mk_logprobs(ctypes.byref(_args(**over)), None) == code
    assert mk.lib().mk_logprobs(None, None) == mk.ERR_INVALID_ARG


def test_the_loops_settings():
    model = types.SimpleNamespace(config=types.SimpleNamespace(vocab=10), check=lambda: None)
    for bad in (-1, 11, 65):
        with pytest.raises(ValueError):
            sampling.SampledLoop(model, None, [1, 2], [0, 0], 10, device="cpu", logprobs=bad)
    loop = sampling.SampledLoop(model, None, [1, 2], [0, 0], 10, device="cpu", logprobs=3)
    assert [tuple(x.shape) for x in loop.logprobs()] == [(2, 0), (2, 0), (2, 0, 3), (2, 0, 3)]
    with pytest.raises(ValueError):
        sampling.SampledLoop(model, None, [1, 2], [0, 0], 10, device="cpu").logprobs()


# ---------------------------------------------------------------- on the GPU

@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,V,given,top", [
    (1, 1, 1, 1), (1, 2, 2, 2), (3, 7, 1, 5), (1, 33, 1, 0), (5, 64, 3, 64), (2, 1000, 1, 20), (7, 4097, 2, 33),
    (1, 32000, 1, 5), (40, 8191, 1, 1), (2, 151936, 1, 64), (200, 2500, 1, 20), (500, 300, 1, 7), (170, 40001, 1, 5),
])
def test_against_the_definition(dtype, R, V, given, top):
    g = torch.Generator(device="cuda").manual_seed(R + V)
    x = (torch.randn((R, V), generator=g, device="cuda") * 3).to(dtype)
    tokens = torch.randint(0, V, (R, given), generator=g, device="cuda").to(torch.int32)
    check(x, tokens, top)
    T = 0.3 + 2 * torch.rand((R,), generator=g, device="cuda")
    check(x, tokens[:, 0].contiguous(), top, T)
    check(x, None, top, T)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "one", "few", "steps", "huge", "saw"])
@pytest.mark.parametrize("R,V", [(1, 5000), (3, 70001), (300, 3001)])
def test_orders_and_ties(dtype, kind, R, V):
    i = torch.arange(V, device="cuda", dtype=torch.float32).expand(R, V)
    x = {"equal": lambda: torch.full((R, V), 1.5, device="cuda"), "rising": lambda: i * 1e-3, "falling": lambda: -i * 1e-3,
         "one": lambda: torch.where(i == V - 1, 40.0, 0.0), "few": lambda: torch.where(i % 997 == 5, 7.0, -math.inf),
         "steps": lambda: (i % 17).floor(), "huge": lambda: (i % 23 - 11) * (5000.0 if dtype == torch.float16 else 1e30),
         "saw": lambda: (i % 1024) * 0.01 + i * 1e-5}[kind]().to(dtype).contiguous()
    tokens = torch.full((R, 1), V - 1, dtype=torch.int32, device="cuda")
    if kind == "huge":  # everything but the largest ones has weight 0
        got, h, ids, best = sampling.logprobs(x, tokens, top=20)
        n = (x[0].float() == x[0].float().max()).sum().item()
        assert torch.allclose(h, torch.full_like(h, math.log(n)), rtol=1e-6)
        assert torch.equal(ids.long(), x.float().sort(dim=-1, descending=True, stable=True).indices[:, :20])
        return
    check(x, tokens, 20)


@gpu
@pytest.mark.parametrize("V", [100, 50001])
def test_masks_and_rows_without_a_distribution(V):
    x = torch.randn((9, V), device="cuda")
    x[0] = -math.inf                      # nothing unmasked
    x[1, V // 2] = math.nan
    x[2, V - 1] = math.inf
    x[3, 3:] = -math.inf                  # three tokens left
    x[4, :] = -math.inf
    x[4, 17] = -3.0                       # one left
    x[5, ::2] = -math.inf
    tokens = torch.tensor([[0, 1], [0, 1], [0, 1], [2, 50], [17, 16], [1, 0], [-1, V], [2 ** 31 - 1, 0], [5, 5]],
                          dtype=torch.int32, device="cuda")
    T = torch.ones((9,), device="cuda")
    T[7] = 0.0
    for temperature in (None, T):
        got, h, ids, best = sampling.logprobs(x, tokens, top=4, temperature=temperature)
        bad = [0, 1, 2] + ([7] if temperature is not None else [])
        for r in range(9):
            if r in bad:
                assert got[r].isnan().all() and h[r].isnan() and (ids[r] == -1).all() and best[r].isnan().all()
        assert got[3, 1] == -math.inf and not got[3, 0].isnan()
        assert set(ids[3, :3].tolist()) == {0, 1, 2} and ids[3, 3] == 3 and best[3, 3] == -math.inf
        assert got[4].tolist() == [0.0, -math.inf] and h[4] == 0.0
        assert ids[4].tolist() == [17, 0, 1, 2] and best[4].tolist() == [0.0] + [-math.inf] * 3
        assert got[5, 1] == -math.inf and (ids[5] % 2 == 1).all()
        assert got[6].isnan().all() and not h[6].isnan()
        assert got[8, 0] == got[8, 1]
    T[:] = torch.tensor([1, 1, 1, -1.0, math.nan, math.inf, 1, 1, 1e-30], device="cuda")
    got, h, ids, best = sampling.logprobs(x, tokens, top=2, temperature=T)
    assert got[3].isnan().all() and ids[4].tolist() == [-1, -1]
    # an infinite temperature: all unmasked tokens alike; a tiny one: the largest takes all
    assert abs(h[5] - math.log(V // 2)) < 1e-4 and torch.allclose(best[5], torch.full_like(best[5], -math.log(V // 2)))
    assert best[8, 0] == 0.0 and h[8] == 0.0


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_alignment(dtype):
    wide = torch.randn((6, 3005), device="cuda").to(dtype)
    for x in (wide[:, 1:], wide[:, 3:2998], wide[::2, 5:], wide[:1].expand(4, -1), wide.reshape(-1)[1:-4].view(1, -1)):
        check(x, torch.full((x.shape[0],), 7, dtype=torch.int32, device="cuda"), 9)


@gpu
def test_equal_inputs_equal_outputs_captured_and_on_streams():
    x = torch.randn((3, 90001), device="cuda").half()  # many ties
    tokens = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    first = sampling.logprobs(x, tokens, top=50)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, sampling.logprobs(x, tokens, top=50)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sampling.logprobs(x, tokens, top=50)
    x.copy_(torch.randn_like(x))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, sampling.logprobs(x, tokens, top=50)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sampling.logprobs(x, tokens, top=50, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(out, got))


@gpu
def test_nothing_to_do_and_refusals():
    x = torch.randn((3, 50), device="cuda")
    tok = torch.zeros((3,), dtype=torch.int32, device="cuda")
    a, h, ids, best = sampling.logprobs(x[:0], tok[:0], top=3)
    assert a.shape == (0,) and h.shape == (0,) and ids.shape == (0, 3) and best.shape == (0, 3)
    a, h, ids, best = sampling.logprobs(x, torch.zeros((3, 0), dtype=torch.int32, device="cuda"))
    assert a.shape == (3, 0) and ids.shape == (3, 0) and not h.isnan().any()
    for args, kw in (((x.double(), tok), {}), ((x[0], tok), {}), ((x.cpu(), tok.cpu()), {}), ((x, tok.long()), {}),
                     ((x, tok[:2]), {}), ((x, tok.cpu()), {}), ((x, tok), dict(top=51)), ((x, tok), dict(top=-1)),
                     ((x, tok), dict(temperature=tok)), ((x.t(), tok), {}), ((x, tok[0]), {})):
        with pytest.raises(ValueError):
            sampling.logprobs(*args, **kw)
    with pytest.raises(mk.MKError):
        sampling.logprobs(torch.randn((1, 100), device="cuda"), tok[:1], top=65)


@gpu
def test_a_loop_keeps_its_tokens_probabilities():
    """The decode loop's record against the definition on the step's own logits; without it the tokens are the same."""
    from moe_decode_megakernel_02_gb300 import workload
    from synth import configs
    cfg = configs.TINY
    runs = []
    for top in (None, 3):
        model = workload.load_synthetic(cfg, max_batch=2, max_tokens_per_seq=1, max_ctx=cfg["ctx"] + 8)
        kv = mk.KVCache(model, 2, cfg["ctx"] + 8)
        workload.prefill(kv, cfg, cfg["ctx"])
        loop = sampling.SampledLoop(model, kv, [3, 5], [cfg["ctx"]] * 2, cfg["vocab"], temperature=0.7,
                                    generator=torch.Generator(device="cuda").manual_seed(1), logprobs=top)
        kept = []
        for _ in range(4):
            drawn = loop.step()
            kept.append((loop.logits.clone(), drawn))
        runs.append(loop.tokens())
        if top is None:
            continue
        logp, h, ids, best = loop.logprobs()
        assert logp.shape == h.shape == (2, 4) and ids.shape == best.shape == (2, 4, 3)
        for i, (x, drawn) in enumerate(kept):
            want, entropy, _ = expected(x, None)
            assert torch.allclose(logp[:, i].double(), want.gather(1, drawn[:, None].long())[:, 0].cpu(), atol=1e-5)
            assert torch.allclose(h[:, i].double(), entropy.cpu(), atol=1e-5)
            assert torch.equal(ids[:, i].long(), x.sort(dim=-1, descending=True, stable=True).indices[:, :3].cpu())
    assert runs[0] == runs[1]


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("top", [1, 2, 7, 32, 33, 64])
@pytest.mark.parametrize("rows,V", [(3, 1000), (2, 32000), (200, 40011)])
def test_rows_full_of_nan(dtype, top, rows, V):
    """NaNs of many threads at once, also in later rounds with logits that rise, beside rows without any."""
    g = torch.Generator("cuda").manual_seed(11)
    x = torch.randn(rows, V, device="cuda", generator=g)
    x[0] = torch.arange(V, device="cuda") * (64.0 / V)
    x[0][torch.rand(V, device="cuda", generator=g) < 0.3] = math.nan
    x[1] = torch.arange(V, device="cuda") * (64.0 / V)
    x[1, V // 2::37] = math.nan
    x = x.to(dtype)
    tokens = torch.arange(rows, device="cuda", dtype=torch.int32)
    got, h, ids, best = sampling.logprobs(x, tokens, top=top)
    assert got[:2].isnan().all() and h[:2].isnan().all() and (ids[:2] == -1).all() and best[:2].isnan().all()
    if rows > 2:
        check(x[2:], tokens[2:], top)
