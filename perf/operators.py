"""Cases of the operators on paged caches and logits: what a serving loop runs around its own layers.

    write   quantises new K and V rows as they go into a paged cache (8-bit codes, one 32-bit scale a row)
    read    reads positions of such a cache back as 16-bit rows
    attend  attention of one or a few new tokens a sequence over the pages of a batch, whose first
            positions may be shared by all; scores may be capped by a tanh, biased by distance, and
            masked before a document's start
    sample  draws one token a row from logits (temperature, top-k, top-p, min-p) with given random numbers

Each is stated here in plain torch operations; with `own` set the same inputs go through the framework's
calls. A cache is [pages, kv heads, page size, head dim] with scales [pages, kv heads, page size]; position j
of sequence b is row j % page size of page table[b, j // page size].
"""
import math

import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}
CODES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
FLOATS = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TINY = 2.0 ** -126  # the least normal 32-bit number: a row of zeros gets this scale


def _write(name, fmt, dtype, B, T, H, D, ps, ragged):
    return {"name": name, "op": "write", "fmt": fmt, "dtype": dtype, "B": B, "T": T, "H": H, "D": D, "ps": ps,
            "ragged": ragged}


def _read(name, fmt, dtype, B, T, H, D, ps, ragged):
    return dict(_write(name, fmt, dtype, B, T, H, D, ps, ragged), op="read")


def _attend(name, fmt, dtype, B, T, Hq, H, D, L, ps, shared=0, cap=0.0, alibi=False, starts=False, pad=False):
    return {"name": name, "op": "attend", "fmt": fmt, "dtype": dtype, "B": B, "T": T, "Hq": Hq, "H": H, "D": D,
            "L": L, "ps": ps, "shared": shared, "cap": cap, "alibi": alibi, "starts": starts, "pad": pad}


def _sample(name, dtype, R, V, mode):
    return {"name": name, "op": "sample", "dtype": dtype, "R": R, "V": V, "mode": mode}


def listed():
    return [
        # the new token of each of 8 sequences of the mid model (4 kv heads of 128): once a layer and step, latency counts
        _write("write_step_e4m3", "e4m3", "bf16", 8, 1, 4, 128, 64, False),
        # the prompts of a batch of 16, up to 4096 tokens each, dense model's 8 kv heads: bandwidth
        _write("write_prompts_int8", "int8", "bf16", 16, 4096, 8, 128, 64, True),
        # an odd, ragged chunk of small heads from a 16-bit float model into small pages
        _read("read_chunk_int8", "int8", "fp16", 5, 777, 2, 64, 16, True),
        # a parked batch of prompts comes back as bf16 rows
        _read("read_prompts_e4m3", "e4m3", "bf16", 16, 4096, 8, 128, 64, False),
        # one user, the mid model's heads at its context: the smallest attention call
        _attend("attend_one_bf16", "bf16", "bf16", 1, 1, 16, 4, 128, 4096, 64),
        # a verify block of 7 tokens for 8 sequences at 8192 positions, capped scores
        _attend("attend_verify_e4m3_cap", "e4m3", "bf16", 8, 7, 16, 4, 128, 8192, 64, cap=30.0),
        # a serving batch of 64 ragged long contexts in 8 bits, dense model's heads: cache bandwidth
        _attend("attend_batch_e4m3", "e4m3", "bf16", 64, 1, 40, 8, 128, 32768, 64),
        # 64 conversations on one 16384-token prefix, each with up to 1024 tokens of its own
        _attend("attend_shared_bf16", "bf16", "bf16", 64, 1, 40, 8, 128, 17408, 64, shared=16384),
        # odd lengths, small pages and heads, distance bias, documents that start late, a padded sequence
        _attend("attend_docs_int8", "int8", "fp16", 13, 2, 8, 2, 64, 2611, 16, alibi=True, starts=True, pad=True),
        # one row of the mid model's vocabulary, all filters on
        _sample("sample_one_fp32", "fp32", 1, 32000, "mixed"),
        # a batch of 32 rows of the deep model's vocabulary, top-p alone
        _sample("sample_top_p_fp32", "fp32", 32, 64000, "top_p"),
        # a batch of 256 rows of the dense model's vocabulary, every row with its own settings
        _sample("sample_batch_bf16", "bf16", 256, 151936, "mixed"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend", "sample", "sample"])
    ps = rng.choice([16, 32, 64, 128])
    H, D = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 256])
    if op in ("write", "read"):
        B, fmt = _log(rng, 1, 32), rng.choice(["e4m3", "int8"])
        T = _log(rng, 1, max(1, 67108864 // (B * H * D)))
        c = _write("", fmt, rng.choice(["bf16", "fp16", "fp32"]), B, min(T, 20000), H, D, ps, rng.random() < 0.5)
        c["op"] = op
    elif op == "attend":
        B, T = _log(rng, 1, 96), rng.choice([1, 1, 1, 2, 4, 7])
        fmt = rng.choice(["bf16", "e4m3", "int8"])
        G = rng.choice([1, 2, 4, 5, 8])
        L = min(_log(rng, 1, 65536), max(1, 536870912 // (B * H * D * (2 if fmt == "bf16" else 1))),
                max(1, 671088640 // (B * T * H * G * 64)))
        shared = 0
        if B > 1 and L > 2 * ps and rng.random() < 0.35:
            shared = rng.randrange(1, L // ps) * ps
        c = _attend("", fmt, rng.choice(["bf16", "bf16", "fp16"]), B, T, H * G, H, D, L, ps, shared=shared,
                    cap=rng.choice([0.0, 0.0, 20.0, 50.0]), alibi=rng.random() < 0.3,
                    starts=shared == 0 and rng.random() < 0.3, pad=B > 2 and rng.random() < 0.3)
    else:
        R = _log(rng, 1, 256)
        c = _sample("", rng.choice(["fp32", "bf16", "fp16"]), R, _log(rng, 100, 151936),
                    rng.choice(["plain", "top_k", "top_p", "min_p", "mixed"]))
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _spread(n, most, least):
    """n whole numbers of [least, most], spread unevenly, the first of them `most`."""
    return [most - (i * 2654435761 >> 5) % (most - least + 1) if i else most for i in range(n)]


def _counts(case):
    return _spread(case["B"], case["T"], case["T"] // 4) if case["ragged"] else [case["T"]] * case["B"]


def _lens(case):
    mine = case["L"] - case["shared"]
    lens = [case["shared"] + n for n in _spread(case["B"], mine, min(mine, max(1, mine // 4)))]
    if case["pad"]:
        lens[-1] = 0
    return lens


def _starts(case):
    return [n // 3 for n in _lens(case)] if case["starts"] else [0] * case["B"]


def _quantised(x, fmt):
    """Codes and scales of the rows of x: the scale is the row's largest magnitude over the format's."""
    x = x.float()
    if fmt == "bf16":
        return x.to(torch.bfloat16), None
    largest = x.abs().amax(-1)
    # a true quotient: torch multiplies by the reciprocal of a plain number
    scale = (largest / torch.full_like(largest, QMAX[fmt])).clamp_min(TINY)
    y = x / scale[..., None]
    return (y.round().to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)), scale


def _random_cache(g, fmt, pages, H, ps, D):
    codes = torch.empty((pages, H, ps, D), dtype=CODES[fmt], device="cuda")
    scales = None if fmt == "bf16" else torch.empty((pages, H, ps), device="cuda")
    for i in range(0, pages, 2048):
        x = torch.randn((min(2048, pages - i), H, ps, D), generator=g, device="cuda", dtype=torch.bfloat16)
        c, s = _quantised(x, fmt)
        codes[i:i + 2048] = c
        if s is not None:
            scales[i:i + 2048] = s
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    s = {"case": case, "op": case["op"]}
    if case["op"] == "sample":
        R, V, mode = case["R"], case["V"], case["mode"]
        x = torch.randn((R, V), generator=g, device="cuda") * 2.5
        # a few tokens stand out, as a trained model's do
        at = torch.randint(0, V, (R, 12), generator=g, device="cuda")
        x.scatter_add_(1, at, 8 + 4 * torch.rand((R, 12), generator=g, device="cuda"))

        def pick(values, dtype, on):
            i = torch.randint(0, len(values), (R,), generator=g, device="cuda")
            v = torch.tensor(values, dtype=dtype, device="cuda")
            return v[i] if on else torch.full((R,), values[0], dtype=dtype, device="cuda")

        mixed = mode == "mixed"
        s.update(logits=x.to(FLOATS[case["dtype"]]),
                 u=torch.rand((R,), generator=g, device="cuda"),
                 temperature=pick([1.0, 0.7, 0.9, 1.3] + ([0.0] if mixed else []), torch.float32, True),
                 top_k=pick([0, 50, 20, 200], torch.int32, mixed or mode == "top_k"),
                 top_p=pick([1.0, 0.9, 0.95, 0.6], torch.float32, mixed or mode == "top_p"),
                 min_p=pick([0.0, 0.05, 0.01], torch.float32, mixed or mode == "min_p"))
        return s

    B, T, H, D, ps, fmt = (case[k] for k in ("B", "T", "H", "D", "ps", "fmt"))
    if case["op"] == "attend":
        longest, shared = case["L"], case["shared"] // ps
    else:
        longest, shared = case["T"] + 3 * ps, 0
    cols = -(-longest // ps)
    pages = shared + B * (cols - shared) + 1  # one page that nobody holds
    order = torch.randperm(pages, generator=g, device="cuda")[:pages - 1].to(torch.int32)
    table = torch.empty((B, cols), dtype=torch.int32, device="cuda")
    table[:, :shared] = order[:shared]
    table[:, shared:] = order[shared:].view(B, cols - shared)
    s.update(table=table, ps=ps, fmt=fmt)
    s["k"], s["ks"] = _random_cache(g, fmt, pages, H, ps, D)
    s["v"], s["vs"] = _random_cache(g, fmt, pages, H, ps, D)
    dtype = FLOATS[case["dtype"]]
    if case["op"] == "attend":
        s.update(q=torch.randn((B, T, case["Hq"], D), generator=g, device="cuda").to(dtype), lens=ints(_lens(case)),
                 starts=ints(_starts(case)) if case["starts"] else None, scale=1 / math.sqrt(D))
        if case["alibi"]:
            h = torch.arange(1, case["Hq"] + 1, device="cuda", dtype=torch.float32)
            s["slopes"] = torch.exp2(-8 * h / case["Hq"])
        else:
            s["slopes"] = None
        return s
    s["positions"] = torch.randint(0, 3 * ps + 1, (B,), generator=g, device="cuda").to(torch.int32)
    s["counts"] = ints(_counts(case)) if case["ragged"] else None
    s["dtype"] = dtype
    if case["op"] == "write":
        # a fused projection's output, K and V side by side in each token's row
        kv = torch.randn((B, T, 2, H, D), generator=g, device="cuda").to(dtype)
        s["k_new"], s["v_new"] = kv[:, :, 0], kv[:, :, 1]
    else:
        s["out"] = tuple(torch.zeros((B, T, H, D), dtype=dtype, device="cuda") for _ in range(2))
    return s


# ---------------------------------------------------------------- the plain forms

def _bytes(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _places(s, B, T):
    """Sequence, row, page and row in the page of every new position that counts."""
    t = torch.arange(T, device="cuda")
    if s["counts"] is None:
        b, t = torch.arange(B, device="cuda").repeat_interleave(T), t.repeat(B)
    else:
        b, t = (t < s["counts"][:, None]).nonzero(as_tuple=True)
    pos = s["positions"][b].long() + t
    return b, t, s["table"][b, pos // s["ps"]].long(), pos % s["ps"]


def _plain_write(s):
    B, T = s["k_new"].shape[:2]
    b, t, page, row = _places(s, B, T)
    for new, codes, scales in ((s["k_new"], s["k"], s["ks"]), (s["v_new"], s["v"], s["vs"])):
        c, sc = _quantised(new[b, t], s["fmt"])
        _bytes(codes)[page, :, row] = _bytes(c)
        scales[page, :, row] = sc
    return [s["k"], s["ks"], s["v"], s["vs"]]


def _plain_read(s):
    B, T = s["out"][0].shape[:2]
    b, t, page, row = _places(s, B, T)
    for out, codes, scales in ((s["out"][0], s["k"], s["ks"]), (s["out"][1], s["v"], s["vs"])):
        c = _bytes(codes)[page, :, row].view(codes.dtype).float()
        out[b, t] = (c * scales[page, :, row][..., None]).to(out.dtype)
    return list(s["out"])


def _rows(s, codes, scales, L):
    """[B, L, H, D] in 32 bits: the first L positions of every sequence."""
    j = torch.arange(L, device="cuda")
    page, row = s["table"][:, j // s["ps"]].long(), j % s["ps"]
    x = _bytes(codes)[page, :, row].view(codes.dtype).float()
    return x if scales is None else x * scales[page, :, row][..., None]


def _plain_attend(s):
    q = s["q"]
    B, T, Hq, D = q.shape
    H, L = s["k"].shape[1], s["case"]["L"]
    x = torch.einsum("bthgd,blhd->bhgtl", q.float().view(B, T, H, Hq // H, D), _rows(s, s["k"], s["ks"], L)) * s["scale"]
    cap = s["case"]["cap"]
    if cap > 0:
        x = cap * torch.tanh(x / cap)
    at = s["lens"].long()[:, None] - T + torch.arange(T, device="cuda")  # the position of each new token
    j = torch.arange(L, device="cuda")
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, H, Hq // H, 1, 1) * (at[:, :, None] - j).float()[:, None, None]
    seen = j <= at[:, :, None]
    if s["starts"] is not None:
        seen = seen & (j >= s["starts"][:, None, None])
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.masked_fill(m == -math.inf, 0.0))
    l = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgtl,blhd->bthgd", p / l.masked_fill(l == 0, 1.0), _rows(s, s["v"], s["vs"], L))
    lse = (m + torch.log(l)).squeeze(-1).permute(0, 3, 1, 2).reshape(B, T, Hq)
    return [o.reshape(B, T, Hq, D).to(q.dtype), lse]


def _plain_sample(s):
    """Weights are 32-bit, their sums 64-bit: a token's place in the sum decides, so the sums may not lose it."""
    x = s["logits"].float()
    R, V = x.shape
    temperature = s["temperature"][:, None]
    greedy = temperature <= 0
    z = (x - x.amax(-1, keepdim=True)) / torch.where(greedy, 1.0, temperature)
    w = torch.exp(z)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    rank = torch.arange(V, device="cuda")
    k = torch.where(s["top_k"] > 0, s["top_k"], V)[:, None]
    mass = torch.where(rank < k, ws.double(), 0.0)
    before = mass.cumsum(-1) - mass
    p = torch.where(s["top_p"] < 1, s["top_p"].double(), math.inf)[:, None]
    keep = (rank < k) & (before < p * mass.sum(-1, keepdim=True)) & (ws >= s["min_p"][:, None]) & ~greedy
    keep[:, 0] = True
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    c = torch.where(kept, w.double(), 0.0).cumsum(-1)
    total = c[:, -1:]
    token = (c <= s["u"].double()[:, None] * total).sum(-1)
    prob = w.gather(1, token[:, None]).double() / total
    return [token.to(torch.int32), prob[:, 0].float(), keep.sum(-1).to(torch.int32)]


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    op = s["op"]
    if op == "sample":
        from moe_decode_megakernel_02_gb300 import sampling

        return sampling.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                               top_p=s["top_p"], min_p=s["min_p"], return_details=True)
    cache = s.get("cache")
    if cache is None:  # the handle that a program keeps beside its cache
        from moe_decode_megakernel_02_gb300 import pages

        cache = s["cache"] = pages.Pages(s["k"], s["v"], s["ks"], s["vs"])
    if op == "write":
        cache.write(s["table"], s["positions"], s["k_new"], s["v_new"], counts=s["counts"])
        return [s["k"], s["ks"], s["v"], s["vs"]]
    if op == "read":
        return list(cache.read(s["table"], s["positions"], s["out"][0], s["out"][1], counts=s["counts"]))
    return list(cache.attend(s["table"], s["lens"], s["q"], scale=s["scale"], softcap=s["case"]["cap"],
                             slopes=s["slopes"], starts=s["starts"], shared_len=s["case"]["shared"], return_lse=True))


def run(state):
    if own:
        return _own(state)
    return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend, "sample": _plain_sample}[state["op"]](state)


def work(case):
    if case["op"] == "sample":
        return {"bytes": case["R"] * (case["V"] * FLOATS[case["dtype"]].itemsize + 32), "flops": case["R"] * case["V"] * 4}
    H, D, code = case["H"], case["D"], CODES[case["fmt"]].itemsize
    held = 2 * H * (D * code + (0 if case["fmt"] == "bf16" else 4))  # K and V of one position in the cache
    wide = FLOATS[case["dtype"]].itemsize
    if case["op"] != "attend":
        n = sum(_counts(case))
        return {"bytes": n * (held + 2 * H * D * wide), "flops": n * 2 * H * D * 3}
    lens, T, Hq = _lens(case), case["T"], case["Hq"]
    starts = _starts(case)
    mine = sum(max(0, n - case["shared"] - st) for n, st in zip(lens, starts))
    seen = sum(max(0, n - T + t + 1 - st) for n, st in zip(lens, starts) for t in range(T))
    return {"bytes": (mine + case["shared"]) * held + case["B"] * T * Hq * (2 * D * wide + 4),
            "flops": 4 * D * Hq * seen}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_codes(rows, fmt):
    rows = rows.double()
    scale = rows.abs().amax(-1, keepdim=True).div(QMAX[fmt]).clamp(min=TINY)
    y = rows / scale
    if fmt == "int8":
        return y.round(), scale[..., 0]
    # E4M3: steps of 2^-3 of a value's power of two, of 2^-9 below 2^-6
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (y / step).round() * step, scale[..., 0]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(s)
    ps, table = s["ps"], s["table"].tolist()
    if case["op"] == "attend":
        return _exact_attend(s, case, table)
    first, counts = s["positions"].tolist(), _counts(case)
    if case["op"] == "write":
        outs = []
        for new, codes, scales in ((s["k_new"], s["k"], s["ks"]), (s["v_new"], s["v"], s["vs"])):
            # whole codes are compared as they are: only codes that are numbers of a float type have an error
            c64, s64 = codes.double() if case["fmt"] == "e4m3" else None, scales.double()
            for b in range(case["B"]):
                pos = torch.arange(first[b], first[b] + counts[b])
                pg = torch.tensor([table[b][p // ps] for p in pos.tolist()], dtype=torch.long, device="cuda")
                c, sc = _exact_codes(new[b, :counts[b]], case["fmt"])
                if c64 is not None:
                    c64[pg, :, (pos % ps).cuda()] = c
                s64[pg, :, (pos % ps).cuda()] = sc
            outs += [c64, s64]
        return outs
    outs = []
    for out, codes, scales in ((s["out"][0], s["k"], s["ks"]), (s["out"][1], s["v"], s["vs"])):
        o = out.double()
        for b in range(case["B"]):
            whole = torch.cat([codes[pg].double() * scales[pg].double()[..., None] for pg in table[b]], dim=1)
            o[b, :counts[b]] = whole[:, first[b]:first[b] + counts[b]].transpose(0, 1)
        outs.append(o)
    return outs


def _exact_attend(s, case, table):
    B, T, Hq, H, D, ps = (case[k] for k in ("B", "T", "Hq", "H", "D", "ps"))
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    lens, starts = _lens(case), _starts(case)
    for b in range(B):
        if lens[b] == 0:
            continue
        pg = torch.tensor(table[b][:-(-lens[b] // ps)], dtype=torch.long, device="cuda")

        def head(codes, scales, h):
            x = codes[pg, h].double()
            return (x if scales is None else x * scales[pg, h].double()[..., None]).reshape(-1, D)

        for h in range(H):
            K, V = head(s["k"], s["ks"], h), head(s["v"], s["vs"], h)
            for t in range(T):
                end = lens[b] - T + t + 1
                if end <= starts[b]:
                    continue
                q = s["q"][b, t, h * (Hq // H):(h + 1) * (Hq // H)].double()
                x = (q @ K[starts[b]:end].T) * s["scale"]
                if case["cap"] > 0:
                    x = torch.tanh(x / case["cap"]) * case["cap"]
                if s["slopes"] is not None:
                    far = torch.arange(end - 1 - starts[b], -1, -1, dtype=torch.float64, device="cuda")
                    x = x - s["slopes"][h * (Hq // H):(h + 1) * (Hq // H), None].double() * far
                out[b, t, h * (Hq // H):(h + 1) * (Hq // H)] = torch.softmax(x, -1) @ V[starts[b]:end]
                lse[b, t, h * (Hq // H):(h + 1) * (Hq // H)] = torch.logsumexp(x, -1)
    return [out, lse]


def _exact_sample(s):
    """The probability of the token drawn; the exponent is a 32-bit number by definition."""
    R, V = s["logits"].shape
    probs = torch.empty((R,), dtype=torch.float64, device="cuda")
    for r in range(R):
        x = s["logits"][r].float()
        T, k, p, least, u = (float(s[n][r]) for n in ("temperature", "top_k", "top_p", "min_p", "u"))
        if T <= 0:
            probs[r] = 1.0
            continue
        w = ((x - x.max()) / T).double().exp()
        ids = x.argsort(descending=True, stable=True)
        if k > 0:
            ids = ids[:int(k)]
        if p < 1:
            share = w[ids].cumsum(0) / w[ids].sum()
            ids = ids[:1 + int((share[:-1] < p).sum())]
        ids = ids[(w[ids] >= least) | (ids == ids[0])].sort().values
        share = w[ids].cumsum(0) / w[ids].sum()
        i = int((share <= u).sum().clamp(max=len(ids) - 1))
        probs[r] = w[ids[i]] / w[ids].sum()
    return [None, probs, None]
