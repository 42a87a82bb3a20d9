"""Calls of the operators on latent caches, prompts, rotations and log probabilities as programs make them: the first ones of
a process inside a capture, two at once, expanded inputs, many sequences, the same id twice."""
import os
import subprocess
import sys

import pytest
import torch

from moe_decode_megakernel_02_gb300 import latent, rotary, sampling
from test_latent import check_attend, gpu, ints, make_cache, make_table, queries
from test_prompt import check as check_prompt
from test_prompt import make, starts

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST = """
import torch
from moe_decode_megakernel_02_gb300 import latent, rotary, sampling

def run(graph):
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    B, T, H, L = 3, 2, 16, 1500
    cols = L // 64 + 2
    cache = latent.LatentPages(rand(cols * B, 64, 512), rand(cols * B, 64, 64))
    table = torch.arange(cols * B, dtype=torch.int32, device="cuda").view(B, cols)
    n, q, rows = torch.full((B,), L, dtype=torch.int32, device="cuda"), rand(B, T, H, 192), rand(B, T, 576)
    w, kv = rand(H, 128, 512) / 16, rand(300, H, 256)
    qp, rp = rand(300, H, 192), rand(300, 64)
    at, freq = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda"), rotary.frequencies(64)
    ids = torch.arange(B * T, dtype=torch.int32, device="cuda")
    def calls():
        qr = rotary.rotate(q[..., 128:], n - T, freq)
        cache.write(table, n - T, rows, gain=w[0, 0], inv_freq=freq)
        o = cache.attend(table, n, torch.einsum("bthd,hdr->bthr", q[..., :128], w), qr, 0.07)
        x = torch.einsum("bthr,hdr->bthd", o, w).reshape(B * T, -1)
        p = latent.attend_prompt(qp, kv[..., :128], rp, kv[..., 128:], at, at, 0.07)
        return (x, p) + sampling.logprobs(x, ids, top=5)
    torch.einsum("bthd,hdr->bthr", q[..., :128], w)  # (the library's own first call)
    torch.einsum("bthr,hdr->bthd", rand(B, T, H, 512), w)
    if not graph:
        return calls()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = calls()
    gr.replay()
    return out

a, b = run(True), run(False)
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(a, b)) and bool(torch.isfinite(a[0].float()).all())
print("same")
"""


@gpu
def test_the_first_calls_of_a_process_may_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


@gpu
def test_two_of_each_at_once():
    """Calls of two streams over one cache, prompt and set of logits, many times, each with its own outputs."""
    cache = make_cache(torch.float16, 200, 64)
    table, lens = make_table(3, 60, 200), ints(3800, 64, 1000)
    q, qr = queries(torch.float16, 3, 3, 16)
    nq, nk = [300, 40], [500, 40]
    pq, pk, pr, pv = make(torch.float16, nq, nk, 4)
    qa, ka = starts(nq), starts(nk)
    x = torch.randn((7, 50000), device="cuda")
    ids = torch.arange(7, dtype=torch.int32, device="cuda")
    freq, pos = rotary.frequencies(64), ints(5, 6, 7)

    def calls(stream=None):
        return (cache.attend(table, lens, q, qr, 0.06, stream=stream),
                latent.attend_prompt(pq, pk, pr, pv, qa, ka, 0.06, stream=stream),
                rotary.rotate(qr, pos, freq, stream=stream)) + sampling.logprobs(x, ids, top=9, stream=stream)

    want = calls()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[calls(s) for s in streams] for _ in range(6)]
    torch.cuda.synchronize()
    for both in got:
        for one in both:
            assert all(torch.equal(a, b) for a, b in zip(one, want))


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_expanded_inputs(dtype):
    """Keys and values that all heads share, one query for all sequences, rows of stride 0."""
    nq = [150, 9]
    q, k, r, v = make(dtype, nq, nq, 3)
    at = starts(nq)
    ks, vs, qs = k[:, :1].expand(-1, 3, -1), v[:, :1].expand(-1, 3, -1), q[:, :1].expand(-1, 3, -1)
    out, lse = latent.attend_prompt(qs, ks, r, vs, at, at, 0.07, return_lse=True)
    check_prompt(qs.contiguous(), ks.contiguous(), r, vs.contiguous(), at, at, 0.07, out, lse)
    cache = make_cache(dtype, 20, 16)
    table, lens = make_table(2, 8, 20), ints(100, 128)
    a, b = queries(dtype, 1, 1, 5)
    check_attend(cache, table[:1].expand(2, -1), lens, a.expand(2, 3, -1, -1), b.expand(2, 3, -1, -1), 0.06)
    x = torch.randn((1, 1, 1, 64), device="cuda").to(dtype)
    got = rotary.rotate(x.expand(2, 5, 3, -1), ints(3, 4), rotary.frequencies(64))
    assert torch.equal(got, rotary.rotate(x.repeat(2, 5, 3, 1), ints(3, 4), rotary.frequencies(64)))
    row = torch.randn((1, 1, 576), device="cuda").to(dtype)
    cache.write(table, ints(0, 0), row.expand(2, 7, -1))
    assert torch.equal(cache.latent[table[1, 0].long(), 6], row[0, 0, :512])


@gpu
def test_many_sequences():
    """More sequences than threads of a block, most of them empty or short."""
    g = torch.Generator().manual_seed(2)
    B = 1500
    nq = (torch.randint(0, 40, (B,), generator=g) * (torch.rand(B, generator=g) < 0.1)).tolist()
    nk = [n + (7 if n else 0) for n in nq]
    q, k, r, v = make(torch.bfloat16, nq, nk, 2)
    at, ka = starts(nq), starts(nk)
    out, lse = latent.attend_prompt(q, k, r, v, at, ka, 0.07, return_lse=True)
    check_prompt(q, k, r, v, at, ka, 0.07, out, lse)
    cache = make_cache(torch.bfloat16, 64, 16)
    table = torch.randint(0, 64, (B, 4), generator=g).to(torch.int32).cuda()
    lens = (torch.randint(0, 65, (B,), generator=g) * (torch.rand(B, generator=g) < 0.3)).to(torch.int32).cuda()
    q, qr = queries(torch.bfloat16, B, 1, 8)
    out, lse = cache.attend(table, lens, q, qr, 0.06, return_lse=True)
    some = lens.nonzero().flatten()[:40]
    check_attend(cache, table[some], lens[some].contiguous(), q[some], qr[some], 0.06, given=(out[some], lse[some]))
    assert (out[lens == 0] == 0).all() and (lse[lens == 0] == -float("inf")).all()


@gpu
def test_long_calls_of_few_heads():
    """Whole prompts through the latent cache: more row blocks than SMs, tokens whose block sees parts of many tiles."""
    cache = make_cache(torch.bfloat16, 64, 64)
    table = make_table(1, 60, 64)
    for T, H, n in ((700, 1, 1000), (600, 20, 700), (1300, 2, 1300)):
        q, qr = queries(torch.bfloat16, 1, T, H)
        check_attend(cache, table, ints(n), q, qr, 0.06)


@gpu
@pytest.mark.parametrize("what", ["latent", "value"])
def test_what_some_rows_see_and_is_no_number(what):
    """A later token's latent (or value) that is not finite: the rows before it are as without it, those that see it have no
    number there either."""
    if what == "latent":
        cache = make_cache(torch.bfloat16, 8, 64)
        table, lens = make_table(1, 4, 8), ints(200)
        q, qr = queries(torch.bfloat16, 1, 7, 16)
        want = cache.attend(table, lens, q, qr, 0.06)
        cache.latent[table[0, 196 // 64].long(), 196 % 64, 17] = float("inf")
        got = cache.attend(table, lens, q, qr, 0.06)
        assert torch.equal(got[:, :3], want[:, :3]) and not got[:, 3:, :, 17].isfinite().any()
        return
    q, k, r, v = make(torch.float16, [300], [300], 2)
    at = ints(0, 300)
    want = latent.attend_prompt(q, k, r, v, at, at, 0.07)
    v[177, 1, 5] = float("nan")
    got = latent.attend_prompt(q, k, r, v, at, at, 0.07)
    assert torch.equal(got[:, 0], want[:, 0]) and torch.equal(got[:177, 1], want[:177, 1]) and got[177:, 1, 5].isnan().all()


@gpu
def test_the_same_id_twice_and_far_rows():
    """Logits past 2^31 elements; ids that repeat."""
    R, V = 15000, 151936
    x = torch.empty((R, V), dtype=torch.bfloat16, device="cuda")  # 4.6 GB
    x[-2:] = torch.randn((2, V), device="cuda").bfloat16()
    x[0] = x[-1]
    ids = ints(7, 7, 100, 7).expand(R, 4).contiguous()
    got, h, top, best = sampling.logprobs(x, ids, top=3)
    assert torch.equal(got[0], got[-1]) and got[-1, 0] == got[-1, 1] == got[-1, 3] and torch.equal(top[0], top[-1])
    want = torch.log_softmax(x[-1].double(), 0)
    assert abs(got[-1, 2].double() - want[100]) < 1e-5
