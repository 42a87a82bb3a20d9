"""Cases of the operators around latent attention and of a token's probability: what a serving loop of the
latent-attention models runs beside the decode step.

    rotate    turns part of each query head by its position's angles (one output, the input stays)
    write     appends a layer's compressed rows to a paged cache: the latent part normalised, the rope part
              rotated, both rounded once
    attend    attention of one or a few new tokens a sequence over such a cache, queries and outputs in the
              latent space (the absorbed form)
    prompt    causal attention of whole prompts, or of chunks behind a context, over expanded keys and values
              of a ragged batch (the expanded form)
    logprobs  log probabilities of given tokens, the distribution's entropy and its most probable tokens

Each is stated here in plain torch operations; with `own` set the same inputs go through the framework's
calls. A latent cache is two tensors, [pages, page size, rank] and [pages, page size, rope]; position j of
sequence b is row j % page size of page table[b, j // page size].
"""
import math

import torch

own = False

FLOATS = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
RANK, ROPE, NOPE = 512, 64, 128  # the deep model's latent, its rope part, its heads' other part (and values)


def _rotate(name, dtype, B, T, H, D, first, n, layout, L, theta, factor=1.0):
    return {"name": name, "op": "rotate", "dtype": dtype, "B": B, "T": T, "H": H, "D": D, "first": first, "n": n,
            "layout": layout, "L": L, "theta": theta, "factor": factor}


def _write(name, dtype, rows, B, T, ps, ragged, layout="half"):
    return {"name": name, "op": "write", "dtype": dtype, "rows": rows, "B": B, "T": T, "ps": ps, "ragged": ragged,
            "layout": layout}


def _attend(name, dtype, B, T, H, L, ps, starts=False, pad=False):
    return {"name": name, "op": "attend", "dtype": dtype, "B": B, "T": T, "H": H, "L": L, "ps": ps, "starts": starts,
            "pad": pad}


def _prompt(name, dtype, B, H, T, ctx, ragged):
    return {"name": name, "op": "prompt", "dtype": dtype, "B": B, "H": H, "T": T, "ctx": ctx, "ragged": ragged}


def _logprobs(name, dtype, R, V, given, top, temperature=False):
    return {"name": name, "op": "logprobs", "dtype": dtype, "R": R, "V": V, "given": given, "top": top,
            "temperature": temperature}


def listed():
    return [
        # the rope part of 16 query heads, one new token of 8 sequences: once a layer and step, latency counts
        _rotate("rotate_step", "bf16", 8, 1, 16, NOPE + ROPE, NOPE, ROPE, "half", 8192, 1e4),
        # whole heads of 128 of a batch of prompts, neighbouring pairs, positions stretched for a long context
        _rotate("rotate_prompts", "bf16", 4, 4001, 40, 128, 0, 128, "interleaved", 131072, 5e5, 8.0),
        # the new token of each of 8 sequences: once a layer and step
        _write("write_step", "bf16", "bf16", 8, 1, 64, False),
        # the prompts of a batch of 16, up to 4096 tokens each, from a 32-bit projection: bandwidth
        _write("write_prompts", "bf16", "fp32", 16, 4096, 64, True),
        # one user at the deep model's context: the smallest attention call
        _attend("attend_one", "bf16", 1, 1, 16, 8192, 64),
        # a verify block of 7 tokens for 8 sequences at 8192 positions
        _attend("attend_verify", "bf16", 8, 7, 16, 8192, 64),
        # a serving batch of 64 ragged long contexts: the cache's bandwidth
        _attend("attend_batch", "bf16", 64, 1, 16, 32768, 64),
        # odd lengths and heads, small pages, documents that start late, a padded sequence, a 16-bit float model
        _attend("attend_docs", "fp16", 13, 3, 5, 2611, 16, starts=True, pad=True),
        # one prompt of 8192 tokens of the deep model: matrix products
        _prompt("prompt_long", "bf16", 1, 16, 8192, 0, False),
        # chunks of 9 ragged prompts behind their contexts, a 16-bit float model with few heads
        _prompt("prompt_chunks", "fp16", 9, 5, 531, 1003, True),
        # one row of the mid model's vocabulary, the drawn token and five alternatives
        _logprobs("logprobs_one", "fp32", 1, 32000, 1, 5),
        # 256 rows of the dense model's vocabulary, scored at their own temperatures, 20 alternatives
        _logprobs("logprobs_batch", "bf16", 256, 151936, 2, 20, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "write", "attend", "attend", "attend", "prompt", "prompt", "logprobs", "logprobs"])
    layout = rng.choice(["half", "interleaved"])
    if op == "rotate":
        n = rng.choice([32, 64, 96, 128])
        D = n + rng.choice([0, 0, 16, 64, 128])
        B, H = _log(rng, 1, 32), rng.choice([1, 2, 5, 8, 16, 40])
        T = _log(rng, 1, max(1, min(16384, 67108864 // (B * H * D))))
        c = _rotate("", rng.choice(["bf16", "fp16", "fp32"]), B, T, H, D, rng.choice([0, D - n]), n, layout,
                    _log(rng, 1000, 1000000), rng.choice([1e4, 5e5]), rng.choice([1.0, 1.0, 4.0]))
    elif op == "write":
        B = _log(rng, 1, 32)
        c = _write("", rng.choice(["bf16", "bf16", "fp16"]), rng.choice(["bf16", "fp16", "fp32"]), B,
                   _log(rng, 1, 65536 // B), rng.choice([16, 32, 64, 128]), rng.random() < 0.5, layout)
    elif op == "attend":
        B, T, H = _log(rng, 1, 96), rng.choice([1, 1, 1, 2, 4, 7, 33]), rng.choice([1, 5, 8, 16, 16, 40, 128])
        L = min(_log(rng, 1, 65536), max(1, 2097152 // B), max(1, 33554432 // (B * T * H)))
        c = _attend("", rng.choice(["bf16", "bf16", "fp16"]), B, T, H, L, rng.choice([16, 32, 64, 128]),
                    starts=rng.random() < 0.3, pad=B > 2 and rng.random() < 0.3)
    elif op == "prompt":
        B, H = _log(rng, 1, 16), rng.choice([1, 2, 5, 8, 16])
        T = _log(rng, 1, min(8192, int(math.sqrt(1073741824 // (B * H)))))
        ctx = 0 if rng.random() < 0.5 else rng.randrange(0, max(1, min(16384, 536870912 // (B * H * T)) - T) + 1)
        c = _prompt("", rng.choice(["bf16", "bf16", "fp16"]), B, H, T, ctx, rng.random() < 0.6)
    else:
        c = _logprobs("", rng.choice(["fp32", "bf16", "fp16"]), _log(rng, 1, 256), _log(rng, 100, 151936),
                      rng.choice([1, 1, 3]), rng.choice([0, 1, 5, 20]), rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _spread(n, most, least):
    """n whole numbers of [least, most], spread unevenly, the first of them `most`."""
    return [most - (i * 2654435761 >> 5) % (most - least + 1) if i else most for i in range(n)]


def _counts(case):
    return _spread(case["B"], case["T"], case["T"] // 4) if case["ragged"] else [case["T"]] * case["B"]


def _lens(case):
    lens = _spread(case["B"], case["L"], max(1, case["L"] // 4))
    if case["pad"]:
        lens[-1] = 0
    return lens


def _starts(case):
    return [n // 3 for n in _lens(case)] if case["starts"] else [0] * case["B"]


def _behind(case):
    """The context of each prompt: the positions before its first new token."""
    return _spread(case["B"], case["ctx"], 0) if case["ragged"] else [case["ctx"]] * case["B"]


def _frequencies(n, theta, factor=1.0):
    """Radians a position of the n/2 pairs; `factor` stretches the positions."""
    return theta ** (-torch.arange(0, n, 2, dtype=torch.float64, device="cuda") / n) / factor


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    s = {"case": case, "op": case["op"]}
    dtype = FLOATS[case["dtype"]]
    if case["op"] == "rotate":
        B, T = case["B"], case["T"]
        s["x"] = normal(B, T, case["H"], case["D"], dtype=dtype)
        s["positions"] = torch.randint(0, case["L"], (B,), generator=g, device="cuda").to(torch.int32)
        s["freq"] = _frequencies(case["n"], case["theta"], case["factor"])
        # what a stretched context scales its cosines and sines by
        s["magnitude"] = 1.0 if case["factor"] == 1.0 else 0.1 * math.log(case["factor"]) + 1.0
        return s
    if case["op"] == "logprobs":
        R, V = case["R"], case["V"]
        x = normal(R, V) * 2.5
        # a few tokens stand out, as a trained model's do
        at = torch.randint(0, V, (R, 12), generator=g, device="cuda")
        x.scatter_add_(1, at, 8 + 4 * torch.rand((R, 12), generator=g, device="cuda"))
        s["logits"] = x.to(dtype)
        given = torch.randint(0, V, (R, case["given"]), generator=g, device="cuda")
        given[:, 0] = at[:, 0]  # one of the likely ones, as a drawn token is
        s["tokens"] = given.to(torch.int32)
        s["temperature"] = 0.6 + torch.rand((R,), generator=g, device="cuda") if case["temperature"] else None
        return s
    if case["op"] == "prompt":
        counts, ctx = _counts(case), _behind(case)
        q_at, k_at = [0], [0]
        for n, c in zip(counts, ctx):
            q_at.append(q_at[-1] + n)
            k_at.append(k_at[-1] + n + c)
        H = case["H"]
        s["q"] = normal(q_at[-1], H, NOPE + ROPE, dtype=dtype)
        kv = normal(k_at[-1], H, 2 * NOPE, dtype=dtype)  # the expanding product's output: keys and values of a head
        s.update(k=kv[..., :NOPE], v=kv[..., NOPE:], k_rope=normal(k_at[-1], ROPE, dtype=dtype), q_at=ints(q_at),
                 k_at=ints(k_at), scale=1 / math.sqrt(NOPE + ROPE), most=(max(counts), max(n + c for n, c in zip(counts, ctx))))
        return s

    B, T, ps = case["B"], case["T"], case["ps"]
    longest = case["L"] if case["op"] == "attend" else T + 3 * ps
    cols = -(-longest // ps)
    pages = B * cols + 1  # one page that nobody holds
    s["table"] = torch.randperm(pages, generator=g, device="cuda")[:pages - 1].to(torch.int32).view(B, cols)
    s["ps"] = ps
    s["latent"] = torch.randn((pages, ps, RANK), generator=g, device="cuda", dtype=dtype)
    s["rope"] = torch.randn((pages, ps, ROPE), generator=g, device="cuda", dtype=dtype)
    if case["op"] == "attend":
        s.update(q=normal(B, T, case["H"], RANK, dtype=dtype), q_rope=normal(B, T, case["H"], ROPE, dtype=dtype),
                 lens=ints(_lens(case)), starts=ints(_starts(case)) if case["starts"] else None,
                 scale=1 / math.sqrt(NOPE + ROPE))
        return s
    s["rows"] = normal(B, T, RANK + ROPE, dtype=FLOATS[case["rows"]]) * 3
    s["gain"] = (1 + 0.1 * normal(RANK)).to(dtype)
    s["eps"] = 1e-6
    s["freq"] = _frequencies(ROPE, 1e4)
    s["positions"] = torch.randint(0, 3 * ps + 1, (B,), generator=g, device="cuda").to(torch.int32)
    s["counts"] = ints(_counts(case)) if case["ragged"] else None
    return s


# ---------------------------------------------------------------- the plain forms

def _turned(x, positions, freq, layout, magnitude=1.0):
    """The last dimension of x (32 bits) turned by angles positions * freq; positions broadcasts over x's others."""
    a = positions[..., None].double() * freq
    cos, sin = (a.cos() * magnitude).float(), (a.sin() * magnitude).float()
    if layout == "half":
        n = x.shape[-1] // 2
        x0, x1 = x[..., :n], x[..., n:]
        return torch.cat([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1)
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1).flatten(-2)


def _plain_rotate(s):
    c, x = s["case"], s["x"]
    at = s["positions"][:, None, None] + torch.arange(c["T"], device="cuda")[:, None]
    out = x.clone()
    part = slice(c["first"], c["first"] + c["n"])
    out[..., part] = _turned(x[..., part].float(), at, s["freq"], c["layout"], s["magnitude"]).to(x.dtype)
    return out


def _plain_write(s):
    B, T = s["rows"].shape[:2]
    t = torch.arange(T, device="cuda")
    if s["counts"] is None:
        b, t = torch.arange(B, device="cuda").repeat_interleave(T), t.repeat(B)
    else:
        b, t = (t < s["counts"][:, None]).nonzero(as_tuple=True)
    at = s["positions"][b].long() + t
    page, row = s["table"][b, at // s["ps"]].long(), at % s["ps"]
    x = s["rows"][b, t].float()
    c, r = x[:, :RANK], x[:, RANK:]
    c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + s["eps"]) * s["gain"].float()
    s["latent"][page, row] = c.to(s["latent"].dtype)
    s["rope"][page, row] = _turned(r, at, s["freq"], s["case"]["layout"]).to(s["rope"].dtype)
    return [s["latent"], s["rope"]]


def _softmax(x, seen):
    """Weights and log of the sum over the last dimension of what `seen` leaves; rows that see nothing: 0 and -inf."""
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    w = (x - torch.where(m == -math.inf, torch.zeros_like(m), m)).exp()
    total = w.sum(-1, keepdim=True)
    return w / torch.where(total == 0, torch.ones_like(total), total), (m + total.log()).squeeze(-1)


def _plain_attend(s):
    B, T, H = s["q"].shape[:3]
    L = s["case"]["L"]
    j = torch.arange(L, device="cuda")
    page, row = s["table"][:, j // s["ps"]].long(), j % s["ps"]
    keys = torch.cat([s["latent"][page, row], s["rope"][page, row]], -1).float()  # [B, L, RANK + ROPE]
    q = torch.cat([s["q"], s["q_rope"]], -1).float().reshape(B, T * H, RANK + ROPE)
    x = (torch.matmul(q, keys.transpose(1, 2)) * s["scale"]).view(B, T, H, L)
    last = s["lens"][:, None] - T + torch.arange(T, device="cuda")
    seen = j <= last[..., None]
    if s["starts"] is not None:
        seen &= j >= s["starts"][:, None, None]
    w, lse = _softmax(x, seen[:, :, None])
    out = torch.matmul(w.view(B, T * H, L), keys[..., :RANK]).view(B, T, H, RANK)
    return [out.to(s["q"].dtype), lse]


def _plain_prompt(s):
    """Every sequence padded to the longest."""
    (Tq, Tk), q_at, k_at = s["most"], s["q_at"].long(), s["k_at"].long()
    nq, nk = q_at[1:] - q_at[:-1], k_at[1:] - k_at[:-1]
    i, j = torch.arange(Tq, device="cuda"), torch.arange(Tk, device="cuda")
    qi = (q_at[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    kj = (k_at[:-1, None] + j).clamp(max=s["k"].shape[0] - 1)
    q = s["q"].float()[qi].transpose(1, 2)  # [B, H, Tq, NOPE + ROPE]
    k, v = s["k"].float()[kj].permute(0, 2, 3, 1), s["v"].float()[kj].transpose(1, 2)
    r = s["k_rope"].float()[kj].transpose(1, 2)[:, None]
    x = torch.matmul(q[..., :NOPE], k)
    x += torch.matmul(q[..., NOPE:], r)
    x *= s["scale"]
    seen = j <= (nk - nq)[:, None, None] + i[:, None]
    w, lse = _softmax(x, seen[:, None])
    out = torch.matmul(w, v).transpose(1, 2)  # [B, Tq, H, NOPE]
    b, t = (i < nq[:, None]).nonzero(as_tuple=True)
    return [out[b, t].to(s["q"].dtype), lse.transpose(1, 2)[b, t]]


def _plain_logprobs(s):
    x = s["logits"].float()
    if s["temperature"] is not None:
        x = x / s["temperature"][:, None]
    x = x - x.amax(-1, keepdim=True)
    p = x.exp()
    total = p.sum(-1, keepdim=True)
    logp = x - total.log()
    entropy = -(logp * (p / total)).sum(-1)
    given = logp.gather(1, s["tokens"].long())
    if not s["case"]["top"]:
        return [given, entropy]
    ids = s["logits"].float().sort(dim=-1, descending=True, stable=True).indices[:, :s["case"]["top"]]
    return [given, entropy, ids.to(torch.int32), logp.gather(1, ids)]


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    from moe_decode_megakernel_02_gb300 import latent, rotary, sampling

    c = s["case"]
    if s["op"] == "rotate":
        return rotary.rotate(s["x"], s["positions"], s["freq"], layout=c["layout"], first=c["first"],
                             magnitude=s["magnitude"])
    if s["op"] == "logprobs":
        given, entropy, ids, top = sampling.logprobs(s["logits"], s["tokens"], top=c["top"],
                                                     temperature=s["temperature"])
        return [given, entropy, ids, top] if c["top"] else [given, entropy]
    if s["op"] == "prompt":
        return list(latent.attend_prompt(s["q"], s["k"], s["k_rope"], s["v"], s["q_at"], s["k_at"], s["scale"],
                                         return_lse=True))
    cache = latent.LatentPages(s["latent"], s["rope"])
    if s["op"] == "write":
        cache.write(s["table"], s["positions"], s["rows"], gain=s["gain"], eps=s["eps"], inv_freq=s["freq"],
                    layout=c["layout"], counts=s["counts"])
        return [s["latent"], s["rope"]]
    return list(cache.attend(s["table"], s["lens"], s["q"], s["q_rope"], s["scale"], starts=s["starts"],
                             return_lse=True))


def run(state):
    if own:
        return _own(state)
    return {"rotate": _plain_rotate, "write": _plain_write, "attend": _plain_attend, "prompt": _plain_prompt,
            "logprobs": _plain_logprobs}[state["op"]](state)


def work(case):
    wide = FLOATS[case["dtype"]].itemsize
    if case["op"] == "rotate":
        n = case["B"] * case["T"] * case["H"]
        return {"bytes": 2 * n * case["D"] * wide, "flops": n * case["n"] * 3}
    if case["op"] == "write":
        n = sum(_counts(case))
        return {"bytes": n * (RANK + ROPE) * (FLOATS[case["rows"]].itemsize + wide), "flops": n * (4 * RANK + 3 * ROPE)}
    if case["op"] == "logprobs":
        return {"bytes": case["R"] * (case["V"] * wide + 8 * case["given"] + 8 * case["top"] + 8),
                "flops": case["R"] * case["V"] * 5}
    H = case["H"]
    if case["op"] == "attend":
        lens, starts, B, T = _lens(case), _starts(case), case["B"], case["T"]
        held = sum(max(0, n - st) for n, st in zip(lens, starts))
        seen = sum(max(0, n - T + t + 1 - st) for n, st in zip(lens, starts) for t in range(T))
        return {"bytes": held * (RANK + ROPE) * wide + B * T * H * ((2 * RANK + ROPE) * wide + 4),
                "flops": 2 * (2 * RANK + ROPE) * H * seen}
    counts, ctx = _counts(case), _behind(case)
    new, old = sum(counts), sum(ctx)
    seen = sum(n * c + n * (n + 1) // 2 for n, c in zip(counts, ctx))
    return {"bytes": new * H * ((2 * NOPE + ROPE) * wide + 4) + (new + old) * (2 * H * NOPE + ROPE) * wide,
            "flops": 2 * (2 * NOPE + ROPE) * H * seen}


# ---------------------------------------------------------------- the definitions in 64 bits

def _complex_turned(x, at, freq, layout, magnitude=1.0):
    """x [..., n] in 64 bits: each pair as a complex number times magnitude * exp(i at freq)."""
    n = x.shape[-1]
    z = torch.complex(x[..., :n // 2], x[..., n // 2:]) if layout == "half" else torch.view_as_complex(
        x.reshape(*x.shape[:-1], n // 2, 2).contiguous())
    z = z * torch.polar(torch.full_like(freq, magnitude).expand(*at.shape, -1), at[..., None].double() * freq)
    return torch.cat([z.real, z.imag], -1) if layout == "half" else torch.view_as_real(z).reshape(x.shape)


def _one(q, k, v, scale, first, last):
    """Attention of rows q [n, H, d] over k, v [m, H or 1, d]: row i sees first .. last[i]."""
    x = torch.einsum("nhd,mhd->hnm", q, k.expand(-1, q.shape[1], -1)) * scale
    j = torch.arange(k.shape[0], device="cuda")
    x = x.masked_fill((j < first) | (j > last[:, None]), -math.inf)
    lse = torch.logsumexp(x, -1)
    w = torch.where(lse[..., None] == -math.inf, torch.zeros_like(x), (x - lse[..., None]).exp())
    return torch.einsum("hnm,mhd->nhd", w, v.expand(-1, q.shape[1], -1)), lse.T


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotate":
        out = s["x"].double()
        for b in range(case["B"]):
            at = int(s["positions"][b]) + torch.arange(case["T"], device="cuda")[:, None].expand(-1, case["H"])
            part = out[b, ..., case["first"]:case["first"] + case["n"]]
            part.copy_(_complex_turned(part.clone(), at, s["freq"], case["layout"], s["magnitude"]))
        return out
    if case["op"] == "logprobs":
        outs = [torch.empty(s["tokens"].shape, dtype=torch.float64, device="cuda"),
                torch.empty((case["R"],), dtype=torch.float64, device="cuda"), None,
                torch.empty((case["R"], case["top"]), dtype=torch.float64, device="cuda")]
        for r in range(case["R"]):
            x = s["logits"][r].double()
            if s["temperature"] is not None:
                x = x / s["temperature"][r].double()
            logp = torch.log_softmax(x, 0)
            outs[0][r] = logp[s["tokens"][r].long()]
            outs[1][r] = -(logp.exp() * logp).sum()
            outs[3][r] = logp.sort(descending=True).values[:case["top"]]
        return outs if case["top"] else outs[:2]
    if case["op"] == "prompt":
        q_at, k_at = s["q_at"].tolist(), s["k_at"].tolist()
        outs, lses = [], []
        for b in range(case["B"]):
            keys = slice(k_at[b], k_at[b + 1])
            nq, nk = q_at[b + 1] - q_at[b], k_at[b + 1] - k_at[b]
            k = torch.cat([s["k"][keys], s["k_rope"][keys, None].expand(-1, case["H"], -1)], -1).double()
            v = s["v"][keys].double()
            for i in range(0, nq, 1024):
                n = min(1024, nq - i)
                o, l = _one(s["q"][q_at[b] + i:q_at[b] + i + n].double(), k, v, s["scale"], 0,
                            nk - nq + i + torch.arange(n, device="cuda"))
                outs.append(o)
                lses.append(l)
        return [torch.cat(outs), torch.cat(lses)]
    ps, table = s["ps"], s["table"].long()
    if case["op"] == "attend":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")
        T = case["T"]
        for b, (n, st) in enumerate(zip(_lens(case), _starts(case))):
            if n == 0:
                continue
            pg = table[b, :-(-n // ps)]
            c, r = s["latent"][pg].reshape(-1, RANK)[:n].double(), s["rope"][pg].reshape(-1, ROPE)[:n].double()
            last = n - T + torch.arange(T, device="cuda")
            out[b], lse[b] = _one(torch.cat([s["q"][b], s["q_rope"][b]], -1).double(), torch.cat([c, r], -1)[:, None],
                                  c[:, None], s["scale"], st, last)
        return [out, lse]
    latent, rope = s["latent"].double(), s["rope"].double()
    first = s["positions"].tolist()
    for b, n in enumerate(_counts(case)):
        at = first[b] + torch.arange(n, device="cuda")
        x = s["rows"][b, :n].double()
        norm = x[:, :RANK].norm(dim=-1, keepdim=True)
        c = x[:, :RANK] / (norm.square() / RANK + s["eps"]).sqrt() * s["gain"].double()
        latent[table[b, at // ps], at % ps] = c
        rope[table[b, at // ps], at % ps] = _complex_turned(x[:, RANK:], at, s["freq"], case["layout"])
    return [latent, rope]
