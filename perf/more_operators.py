"""Operators around a verification round's forward pass, as measured cases.

A round verifies ell[r] drafts of request r in rows row0[r] .. row0[r] +
ell[r] of the target's forward pass, at positions len[r] .. len[r] + ell[r] of
its paged cache.  The operators here are what a server adds when contexts get
long and requests bring conditions of their own:

  append     norms and rotation of queries and keys, keys and values into
             8-bit pages, and the blocks they went to read back
  attention  the rows' attention over 8-bit pages
  weigh      the attention weights that a page's tokens get from the round's
             rows, added up per request and page (16-, 8- and 4-bit pages)
  evict      every request's pages down to a budget, least weight first
  logits     penalties for repeated tokens, biases and a grammar's mask on the
             target's logits, and the token counts that they go by

Every operator has a plain form (elementary torch, float32, float64 where a
rounding border or a far position's angle needs it) and the framework's call;
`exact` computes the same from the definition in float64.

8-bit pages hold, of every key/value head: K codes [P/16][D/16][16 tokens]
[16 dims], V codes [P/16][2][32][D/32][8 tokens] (dim e * 32 + i at [i][e]),
then 16 bytes: the scales of the K blocks, from byte 8 on those of the V
blocks.  A code is e4m3 (largest 448); a block of 16 tokens of a head has one
scale 2^(b - 127) for K and one for V, the smallest that brings what the block
holds to at most 448.  Tokens that join a block may raise its scale: the codes
that are there are then rounded again.  The 16-bit and 4-bit layouts are those
of perf/operators.py.
"""

import math

import torch

own = False

EPS = 1e-6
BF16, FP4, FP8 = 1, 2, 4
LOW, HIGH = -117, 119  # exponents that a block's scale may have


# ------------------------------------------------------------------ cases

def _app(name, R, gamma, Hq, Hkv, D, page, ctx, rot, adjacent=False, packed=False, ell="ragged"):
    return dict(name=name, op="append", fmt=FP8, R=R, gamma=gamma, Hq=Hq, Hkv=Hkv, D=D, page=page, ctx=ctx, rot=rot,
                adjacent=adjacent, packed=packed, ell=ell)


def _attn(name, op, fmt, R, gamma, Hq, Hkv, D, page, ctx, window=0, sinks=0, ell="ragged"):
    return dict(name=name, op=op, fmt=fmt, R=R, gamma=gamma, Hq=Hq, Hkv=Hkv, D=D, page=page, ctx=ctx, window=window,
                sinks=sinks, ell=ell)


def _evict(name, R, page, ctx, budget, sinks, recent):
    return dict(name=name, op="evict", R=R, page=page, ctx=ctx, budget=budget, sinks=sinks, recent=recent)


def _logits(name, dtype, R, gamma, V, ell, biases, masked, fresh, ctx):
    return dict(name=name, op="logits", dtype=dtype, R=R, gamma=gamma, V=V, ell=ell, biases=biases, masked=masked,
                fresh=fresh, ctx=ctx)


def listed():
    return [
        # one request, one token: what every decode step of a lone user waits for
        _app("append8_r1_token", 1, 0, 32, 8, 128, 64, 1000, 128, ell="full"),
        # the batched round (128 requests, up to 17 rows each, 56 heads), fused projection rows
        _app("append8_r128_g16_packed", 128, 16, 56, 8, 128, 64, 250, 128, packed=True),
        # one request, one token, a short odd context: latency
        _attn("attn8_r1_token_1023", "attention", FP8, 1, 0, 32, 8, 128, 64, 1023, ell="full"),
        # one token each for 32 requests over long contexts: the bytes of the pages
        _attn("attn8_r32_token_16384", "attention", FP8, 32, 0, 32, 8, 128, 64, 16384, ell="full"),
        # the batched round over ragged contexts up to 16384
        _attn("attn8_r128_g16_16384", "attention", FP8, 128, 16, 56, 8, 128, 64, 16384),
        # one request, one token: weights of the pages of a 16-bit cache
        _attn("weigh_r1_token_4095", "weigh", BF16, 1, 0, 32, 8, 128, 64, 4095, ell="full"),
        # the batched round's rows over 16-bit pages, ragged contexts up to 8192
        _attn("weigh_r128_g16_8192", "weigh", BF16, 128, 16, 56, 8, 128, 64, 8192),
        # a lone request that grew past its budget
        _evict("evict_r1_4000", 1, 64, 4000, 48, 4, 256),
        # 64 long requests in small pages, with shared prefixes, down to half
        _evict("evict_r64_131072", 64, 16, 131072, 4096, 64, 1024),
        # a small vocabulary in 32 bits: a new request, its first round's tokens, its logits
        _logits("logits_r1_g4_v1024_f32", "f32", 1, 4, 1024, "full", 3, True, True, 200),
        # 32 new requests and one row each of a large vocabulary, no grammar
        _logits("logits_r32_token_v151936", "bf16", 32, 0, 151936, "full", 32, False, True, 4000),
        # the batched round with every draft admitted, a grammar's mask a row
        _logits("logits_r128_g16_v129280", "bf16", 128, 16, 129280, "full", 16, True, False, 2000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["append", "attention", "attention", "weigh", "weigh", "evict", "logits", "logits"])
    if op == "evict":
        page = rng.choice([16, 32, 64, 128])
        R = _log(rng, 1, 64)
        ctx = _log(rng, 1, 131072)
        return _evict(None, R, page, ctx, rng.randint(0, max(1, ctx // page)), rng.choice([0, 4, 64]),
                      rng.choice([0, 1, 100, 1024]))
    R = _log(rng, 1, 128)
    gamma = rng.choice([0, 0, rng.randint(1, 16), rng.randint(1, 64), 16])
    ell = rng.choice(["ragged", "full"])
    if op == "logits":
        gamma = min(gamma, 16)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        V = _log(rng, 1000, min(152000, 140_000_000 // (R * (gamma + 1))))
        return _logits(None, dtype, R, gamma, V, ell, rng.choice([0, 1, 20]), rng.choice([False, True]),
                       rng.choice([False, True]), _log(rng, 1, 4000))
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 7, 8])
    D = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        return _app(None, R, gamma, Hq, Hkv, D, page, _log(rng, 1, 300), rng.choice([0, D // 2, D, D]),
                    rng.choice([False, True]), rng.choice([False, True]), ell)
    fmt = FP8 if op == "attention" else rng.choice([BF16, FP4, FP8])
    # a drawn case stays under the largest listed one: its cache by the tokens it may hold, its products by
    # the rows of a full block
    most = 700_000 * 8 * 128 // (Hkv * D)
    ctx = _log(rng, 1, max(8, min(60_000, most // R, 300_000_000 // (R * (gamma + 1) * Hq))))
    window = rng.choice([0, 0, _log(rng, 1, 4096)])
    return _attn(None, op, fmt, R, gamma, Hq, Hkv, D, page, ctx, window, rng.choice([0, 4, 64]) if window else 0, ell)


# ------------------------------------------------------------------ shapes of a case (host numbers)

def _lens(case):
    """Committed tokens of every request: ragged over a quarter to the whole of ctx."""
    R, ctx = case["R"], case["ctx"]
    return [ctx - int(((r * 0.6180339887498949) % 1.0) * 0.75 * ctx) for r in range(R)]


def _ells(case):
    """Admitted drafts: the whole block, or the few that a scheduler admits, with idle requests among them."""
    R, g = case["R"], case["gamma"]
    if case.get("ell") == "full":
        return [g] * R
    e = [int((g + 1) * ((r * 0.7548776662466927 + 0.31) % 1.0) ** 3) for r in range(R)]
    return [-1 if r % 17 == 16 else e[r] for r in range(R)]


def _up(a, b):
    return -(-a // b)


def _half_bytes(fmt, D):
    """Bytes of one token's key, and of its value, of one head (the least that hold them)."""
    return {BF16: (2 * D, 2 * D), FP4: (D / 2 + D / 32, D / 2 + 4), FP8: (D + 1 / 16, D + 1 / 16)}[fmt]


def _shared(case, r):
    """Pages that request r of an eviction has in common with its left neighbour."""
    lens = _lens(case)
    return _up(min(lens[r], lens[r - 1]), case["page"]) // 4 if r % 4 == 3 else 0


def work(case):
    op = case["op"]
    if op == "evict":
        pages = sum(_up(n, case["page"]) for n in _lens(case))
        return {"bytes": 8 * pages + 4 * pages, "flops": 0}
    ells = _ells(case)
    rows = sum(e + 1 for e in ells)
    if op == "logits":
        R, V = case["R"], case["V"]
        size = 4 if case["dtype"] == "f32" else 2
        b = 2 * rows * V * size + R * V * 2 + (rows * V // 8 if case["masked"] else 0)
        if case["fresh"]:
            b += R * V * 2 + 4 * sum(_lens(case))
        return {"bytes": b, "flops": 6 * rows * V}
    lens = _lens(case)
    Hq, Hkv, D, P = case["Hq"], case["Hkv"], case["D"], case["page"]
    kb, vb = _half_bytes(case["fmt"], D)
    if op == "append":
        held = sum(n % 16 for n, e in zip(lens, ells) if e >= 0)
        return {"bytes": rows * (2 * Hq + 2 * Hkv) * D * 2 + int((rows + held) * Hkv * (2 * (kb + vb) + 4 * D)),
                "flops": rows * (Hq + Hkv) * D * 8}
    W, S = case["window"], case["sinks"]
    tokens = seen = pages = 0
    for n, e in zip(lens, ells):
        if e < 0:
            continue
        for i in range(e + 1):
            p = n + i
            low = max(0, p - W + 1) if W else 0
            seen += p + 1 - low + min(S, low)
        low = max(0, n - W + 1) if W else 0
        tokens += n + e + 1 - low + min(S, low)
        pages += _up(n + e + 1, P)
    if op == "weigh":
        return {"bytes": int(tokens * Hkv * kb) + rows * Hq * (2 * D + 4) + 8 * pages, "flops": 2 * seen * Hq * D}
    return {"bytes": int(tokens * Hkv * (kb + vb)) + rows * Hq * (4 * D + 4), "flops": 4 * seen * Hq * D}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _pool(fmt, n_pages, Hkv, D, P, g):
    """A pool that earlier rounds filled."""
    if fmt == BF16:
        pool = torch.empty(n_pages * Hkv * 2 * P * D, dtype=torch.bfloat16, device="cuda")
        for a in range(0, pool.numel(), 1 << 28):
            pool[a:a + (1 << 28)].normal_(generator=g)
        return pool.view(torch.uint8).view(n_pages, -1)
    a = P * D // 2 if fmt == FP4 else P * D
    size = 2 * a + (P * (D // 32 + 4) if fmt == FP4 else 16)
    pool = torch.empty(n_pages * Hkv * size, dtype=torch.uint8, device="cuda")
    if fmt == FP8:
        for i in range(0, pool.numel(), 1 << 27):  # keys and values whose largest are near the scale's end
            x = torch.randn(min(1 << 27, pool.numel() - i), generator=g, device="cuda", dtype=torch.float16) * 80
            pool[i:i + (1 << 27)] = x.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        pool = pool.view(n_pages, Hkv, size)
        pool[:, :, 2 * a:] = torch.randint(120, 122, (n_pages, Hkv, 16), generator=g, device="cuda", dtype=torch.uint8)
        return pool.view(n_pages, -1)
    for i in range(0, pool.numel(), 1 << 26):
        m = min(1 << 26, pool.numel() - i)
        x = torch.randn(2 * m, generator=g, device="cuda", dtype=torch.float16) * 2.3
        y = x.abs()
        c = (x < 0).to(torch.uint8) * 8
        for t in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
            c += y > t
        c = c.view(m, 2)
        pool[i:i + m] = c[:, 0] + c[:, 1] * 16
    pool = pool.view(n_pages, Hkv, size)
    pool[:, :, a:a + P * D // 32] = torch.randint(124, 127, (n_pages, Hkv, P * D // 32), generator=g, device="cuda",
                                                  dtype=torch.uint8)
    s = torch.rand(n_pages, Hkv, P, generator=g, device="cuda") * 0.3 + 0.3
    pool[:, :, 2 * a + P * D // 32:] = s.view(torch.uint8).view(n_pages, Hkv, 4 * P)
    return pool.view(n_pages, -1)


def _tables(need, max_pages, n_pages, g):
    """Pages in no order: request r holds need[r] of them."""
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(need), max_pages), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += n
    return table


def _row0(ells):
    out, rows = [], 0
    for e in ells:
        out.append(rows)
        rows += e + 1
    return out, rows


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "evict":
        return _prepare_evict(case, g)
    if case["op"] == "logits":
        return _prepare_logits(case, g)
    i32 = dict(dtype=torch.int32, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    R, gamma, Hq, Hkv, D, P, fmt = (case[k] for k in ("R", "gamma", "Hq", "Hkv", "D", "page", "fmt"))
    lens, ells = _lens(case), _ells(case)
    need = [_up(n + e + 1, P) for n, e in zip(lens, ells)]
    max_pages = _up(case["ctx"] + gamma + 1, P)
    n_pages = sum(need) + 5
    row0, rows = _row0(ells)
    s = dict(case=case, rows=rows, max_pages=max_pages, spare=n_pages - 1, length=torch.tensor(lens, **i32),
             ell=torch.tensor(ells, **i32), row0=torch.tensor(row0, **i32),
             table=_tables(need, max_pages, n_pages - 1, g), pool=_pool(fmt, n_pages, Hkv, D, P, g))
    if fmt == FP4:
        v16 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
        s["lut"] = torch.stack([v16.repeat(16), v16.repeat_interleave(16)], -1)
    if case["op"] != "append":
        s["q"] = (1.5 * torch.randn(rows, Hq, D, generator=g, device="cuda")).to(torch.bfloat16)
        s["lse"] = torch.zeros(rows, Hq, dtype=torch.float32, device="cuda")
        if case["op"] == "attention":
            s["out"] = torch.zeros(rows, Hq, D, **bf)
            return s
        # the log-sum that the layer's attention left, and the weights of earlier rounds
        req, mine = _row_of(s)
        z = torch.logsumexp(_scores(s, _keys(s)), -1)
        s["lse"].copy_(z.permute(0, 2, 1, 3).reshape(R, gamma + 1, Hq)[req, mine - s["length"][req]])
        s["first"] = 3 * torch.rand(R, max_pages, generator=g, device="cuda") ** 4
        s["mass"] = torch.zeros_like(s["first"])
        return s
    if case["packed"]:
        x = torch.randn(rows, Hq + 2 * Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
        s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    else:
        s["q"], s["k"], s["v"] = (torch.randn(rows, h, D, generator=g, device="cuda").to(torch.bfloat16)
                                  for h in (Hq, Hkv, Hkv))
    s["wq"], s["wk"] = ((1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2))
    rot = case["rot"]
    s["freq"] = 1e4 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device="cuda") / rot) if rot else None
    s["q_out"] = torch.zeros(rows, Hq, D, **bf)
    s["start"] = s["length"] // 16 * 16
    s["count"] = torch.where(s["ell"] >= 0, s["length"] % 16 + s["ell"] + 1, 0).to(torch.int32)
    s["T"] = gamma + 16
    s["k_read"] = torch.zeros(R, s["T"], Hkv, D, **bf)
    s["v_read"] = torch.zeros(R, s["T"], Hkv, D, **bf)
    return s


def _prepare_evict(case, g):
    R, P = case["R"], case["page"]
    lens = _lens(case)
    need = [_up(n, P) for n in lens]
    MP, N = max(need), _up(sum(need) + 7, 32) * 32
    sizes = [R * MP, N, N // 32, R * MP]
    # one buffer holds the whole state, so that a pass starts from the same one with one copy
    first = torch.zeros(sum(sizes), dtype=torch.int32, device="cuda")
    s = dict(case=case, MP=MP, N=N, first=first, state=torch.zeros_like(first),
             length=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             budget=torch.full((R,), case["budget"], dtype=torch.int32, device="cuda"),
             freed=torch.zeros(R, dtype=torch.int32, device="cuda"))
    table = _tables(need, MP, N, g)
    for r in range(R):
        n = _shared(case, r)
        table[r, :n] = table[r - 1, :n]
    ref = torch.zeros(N, dtype=torch.int32, device="cuda")
    _count(ref, table, 1)
    # few pages get most of the weight, some got none at all
    mass = torch.rand(R, MP, generator=g, device="cuda") ** 8 * 50
    mass[torch.rand(R, MP, generator=g, device="cuda") < 0.05] = 0
    first.copy_(torch.cat([table.flatten(), ref, _free_bits(ref), mass.view(torch.int32).flatten()]))
    s["table"], s["ref"], s["bits"], s["mass"] = s["state"].split(sizes)
    s["table"] = s["table"].view(R, MP)
    s["mass"] = s["mass"].view(torch.float32).view(R, MP)
    return s


def _prepare_logits(case, g):
    i32 = dict(dtype=torch.int32, device="cuda")
    R, gamma, V, nb = case["R"], case["gamma"], case["V"], case["biases"]
    ells, lens = _ells(case), _lens(case)
    row0, rows = _row0(ells)

    def tokens(*shape):  # a few tokens are frequent
        u = torch.rand(shape, generator=g, device="cuda", dtype=torch.float64)
        return (V * u ** 4).to(torch.int32).clamp(max=V - 1)

    s = dict(case=case, rows=rows, ell=torch.tensor(ells, **i32), row0=torch.tensor(row0, **i32),
             x0=tokens(R), x=tokens(R, gamma) if gamma else None)
    x = torch.empty(rows, V, device="cuda").normal_(generator=g) * 2
    x[torch.arange(rows, device="cuda"), tokens(rows).long()] += 6
    s["logits"] = x if case["dtype"] == "f32" else x.to(torch.bfloat16)
    s["out"] = torch.zeros_like(s["logits"])
    del x
    u = torch.rand(3, R, generator=g, device="cuda")
    s["repetition"], s["presence"], s["frequency"] = 1 + 0.5 * u[0], u[1], 0.5 * u[2]
    if nb:
        j = torch.arange(nb, device="cuda")
        s["bias_tok"] = ((tokens(R)[:, None] + 31 * j) % V).to(torch.int32)  # no token twice
        s["bias"] = 4 * torch.randn(R, nb, generator=g, device="cuda")
    else:
        s["bias_tok"] = s["bias"] = None
    s["mask"] = None
    if case["masked"]:
        # rows without a grammar, and rows where it allows a half, an eighth and a 64th of the tokens
        W, k = _up(V, 32), torch.arange(rows, device="cuda") % 4
        m = torch.full((rows, W), -1, **i32)
        for n in range(6):
            word = torch.randint(-2 ** 31, 2 ** 31, (rows, W), generator=g, device="cuda", dtype=torch.int64)
            m &= torch.where((n < torch.tensor([0, 1, 3, 6], device="cuda")[k])[:, None], word, -1).to(torch.int32)
        s["mask"] = m
    s["state"] = torch.zeros(R, V, dtype=torch.int16, device="cuda")
    if case["fresh"]:
        s["prompt"] = tokens(sum(lens))
        at = torch.tensor([0] + lens, device="cuda").cumsum(0)
        s["start"], s["count"] = at[:-1].to(torch.int32), torch.tensor(lens, **i32)
        # the round before: its anchors and drafts, and how many of them were kept
        s["x0_before"], s["x_before"] = tokens(R), tokens(R, gamma) if gamma else None
        s["n_acc"] = torch.tensor([int((e + 1) * ((r * 0.5698402909980532) % 1.0)) for r, e in enumerate(ells)], **i32)
    else:
        seen = torch.zeros(R, V, dtype=torch.int32, device="cuda")
        for _ in range(2):  # of the prompt: a flag; of the answer so far: a count
            n = case["ctx"] // 2 + 1
            seen.scatter_add_(1, tokens(R, n).long(), torch.ones(R, n, **i32))
            s["state"] += torch.where(seen > 0, -32768, 0).to(torch.int16) if _ == 0 else seen.to(torch.int16)
            seen.zero_()
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return {"append": _run_append, "attention": _run_attention, "weigh": _run_weigh, "evict": _run_evict,
            "logits": _run_logits}[s["case"]["op"]](s)


def _run_append(s):
    c = s["case"]
    if own:
        from semi_ar_draft_round_amd import binding as B
        B.dspark_cache_append(s["q"], s["k"], s["v"], s["pool"], s["table"], s["length"], s["ell"], c["gamma"],
                              fmt=c["fmt"], page=c["page"], wq=s["wq"], wk=s["wk"], eps=EPS, freq=s["freq"],
                              adjacent=c["adjacent"], row0=s["row0"], q_out=s["q_out"])
        B.dspark_cache_read(s["pool"], s["table"], s["start"], s["count"], s["T"], fmt=c["fmt"], page=c["page"],
                            heads_kv=c["Hkv"], dim=c["D"], k=s["k_read"], v=s["v_read"])
    else:
        _plain_append(s)
        _plain_read(s)
    return {"q": s["q_out"], "k": s["k_read"], "v": s["v_read"]}


def _run_attention(s):
    c = s["case"]
    if own:
        from semi_ar_draft_round_amd import binding as B
        B.dspark_cache_attention(s["q"], s["pool"], s["table"], s["length"], s["ell"], c["gamma"], fmt=c["fmt"],
                                 page=c["page"], heads_kv=c["Hkv"], window=c["window"], sinks=c["sinks"],
                                 row0=s["row0"], out=s["out"], lse=s["lse"])
    else:
        _plain_attention(s)
    return {"out": s["out"], "lse": s["lse"]}


def _run_weigh(s):
    c = s["case"]
    s["mass"].copy_(s["first"])
    if own:
        from semi_ar_draft_round_amd import binding as B
        B.dspark_cache_weigh(s["q"], s["lse"], s["pool"], s["table"], s["length"], s["ell"], c["gamma"], s["mass"],
                             keep=0.75, fmt=c["fmt"], page=c["page"], heads_kv=c["Hkv"], window=c["window"],
                             sinks=c["sinks"], row0=s["row0"])
    else:
        _plain_weigh(s)
    return {"mass": s["mass"]}


def _run_evict(s):
    c = s["case"]
    s["state"].copy_(s["first"])
    if own:
        from semi_ar_draft_round_amd import binding as B
        B.dspark_cache_evict(s["table"], s["length"], s["ref"], s["bits"], s["mass"], s["budget"], page=c["page"],
                             sinks=c["sinks"], recent=c["recent"], freed=s["freed"])
    else:
        _plain_evict(s)
    return {k: s[k] for k in ("table", "ref", "bits", "mass", "freed")}


def _run_logits(s):
    c = s["case"]
    if own:
        from semi_ar_draft_round_amd import binding as B
        if c["fresh"]:
            B.dspark_logits_prompt(s["state"], s["prompt"], s["start"], s["count"])
            B.dspark_logits_commit(s["state"], s["ell"], s["n_acc"], s["x0_before"], s["x_before"])
        B.dspark_logits(s["logits"], s["state"], s["ell"], c["gamma"], s["x0"], s["x"], row0=s["row0"],
                        repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
                        bias_tok=s["bias_tok"], bias=s["bias"], mask=s["mask"], out=s["out"])
    else:
        if c["fresh"]:
            _plain_history(s)
        _plain_logits(s)
    return {"out": s["out"], "state": s["state"]} if c["fresh"] else {"out": s["out"]}


# ------------------------------------------------------------------ plain forms

def _pages(fmt, pool, Hkv, P, D):
    """Views of the pages: 16 bits K [n, Hkv, P/16, D/8, 16, 8] and V [n, Hkv, P/16, 2, D, 8]; 4 bits K codes,
    K scales, V codes, V scales; 8 bits K codes, V codes, the scales of K's blocks and of V's."""
    if fmt == BF16:
        x = pool.view(torch.bfloat16).view(-1, Hkv, 2, P // 16, 16 * D)
        return x[:, :, 0].unflatten(-1, (D // 8, 16, 8)), x[:, :, 1].unflatten(-1, (2, D, 8))
    x = pool.view(pool.shape[0], Hkv, -1)
    if fmt == FP8:
        a = P * D
        return (x[:, :, :a].unflatten(-1, (P // 16, D // 16, 16, 16)),
                x[:, :, a:2 * a].unflatten(-1, (P // 16, 2, 32, D // 32, 8)),
                x[:, :, 2 * a:2 * a + P // 16], x[:, :, 2 * a + 8:2 * a + 8 + P // 16])
    a, b = P * D // 2, P * D // 2 + P * D // 32
    return (x[:, :, :a].unflatten(-1, (P // 16, D // 32, 16, 16)), x[:, :, a:b].unflatten(-1, (P, D // 32)),
            x[:, :, b:b + a].unflatten(-1, (P // 16, 2, 32, D // 32, 4)), x[:, :, b + a:].view(torch.float32))


def _values8(codes):
    return codes.view(torch.float8_e4m3fn).to(torch.float32)


def _codes8(x):
    """e4m3 codes of float64 x, nearest, ties to the even code, at most 448."""
    a = x.abs()
    step = torch.exp2((torch.frexp(a)[1].double() - 1).clamp(min=-6) - 3)
    a = (torch.round(a / step) * step).clamp(max=448)
    return torch.copysign(a, x).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)


def _row_of(s):
    """The request and the position of every packed row."""
    row = torch.arange(s["rows"], dtype=torch.int32, device="cuda")
    req = torch.searchsorted(s["row0"], row, right=True) - 1
    return req, (s["length"][req] + row - s["row0"][req]).long()


def _norm_rotate(x, w, pos, s, real):
    c = s["case"]
    x = x.to(real)
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.to(real)
    rot = c["rot"]
    if not rot:
        return x
    angle = pos[:, None].double() * s["freq"]
    cos, sin = torch.cos(angle).to(real)[:, None], torch.sin(angle).to(real)[:, None]
    if c["adjacent"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _requantise(x, codes, scale, new, old):
    """New codes and scale bytes of blocks [R, NB]: x [R, NB, 16, Hkv, D] where `new` [R, NB, 16], the codes that
    are there where `old`; others stay.  scale [R, NB, Hkv]: the bytes that are there."""
    top = torch.where(new[..., None, None], x, 0).abs().amax((2, 4))
    m, e = torch.frexp(top)
    e = torch.where(top > 0, torch.where(m <= 0.875, e - 9, e - 8), LOW).clamp(LOW, HIGH)
    before = scale.int() - 127
    e = torch.where(old.any(-1)[..., None], torch.maximum(e, before), e)
    at = lambda n: n[:, :, None, :, None].double()
    y = torch.where(new[..., None, None], x, _values8(codes).double() * torch.exp2(at(before)))
    y = _codes8(y * torch.exp2(-at(e)))
    write = new | (old & new.any(-1, keepdim=True))
    return (torch.where(write[..., None, None], y, codes),
            torch.where(new.any(-1)[..., None], (e + 127).to(torch.uint8), scale))


def _plain_append(s):
    c = s["case"]
    Hkv, P, D, n = c["Hkv"], c["page"], c["D"], c["gamma"] + 1
    _, pos = _row_of(s)
    s["q_out"].copy_(_norm_rotate(s["q"], s["wq"], pos, s, torch.float32))
    k = _norm_rotate(s["k"], s["wk"], pos, s, torch.float64)
    # the blocks of 16 tokens that a request's rows can touch
    L = s["length"][:, None].long()
    first = L // 16 * 16 + 16 * torch.arange((n + 30) // 16, device="cuda")                # [R, NB]
    t = first[..., None] + torch.arange(16, device="cuda")                                 # [R, NB, 16]
    new = (t >= L[..., None]) & (t <= (L + s["ell"][:, None])[..., None])
    old = t < L[..., None]
    row = torch.where(new, s["row0"][:, None, None] + t - L[..., None], 0)
    page = s["table"].gather(1, (first // P).clamp(max=s["max_pages"] - 1)).long()
    page = torch.where(new.any(-1), page, s["spare"])                                      # nothing new: aside
    blk = first % P // 16
    kc, vc, ks, vs = _pages(FP8, s["pool"], Hkv, P, D)
    codes = kc[page, :, blk].transpose(-2, -3).flatten(-2).transpose(2, 3)                 # [R, NB, 16, Hkv, D]
    codes, scale = _requantise(k[row], codes, ks[page, :, blk], new, old)
    kc[page, :, blk] = codes.transpose(2, 3).unflatten(-1, (D // 16, 16)).transpose(-2, -3)
    ks[page, :, blk] = scale
    # V: [R, NB, Hkv, 2, 32, E, 8] <-> [R, NB, 16, Hkv, D]
    codes = vc[page, :, blk].movedim(-1, 4).transpose(-1, -2).flatten(-2).flatten(3, 4).transpose(2, 3).contiguous()
    codes, scale = _requantise(s["v"][row].double(), codes, vs[page, :, blk], new, old)
    codes = codes.transpose(2, 3).unflatten(3, (2, 8)).unflatten(-1, (D // 32, 32)).transpose(-1, -2).movedim(4, -1)
    vc[page, :, blk] = codes
    vs[page, :, blk] = scale


def _dense(s, page, values=True):
    """K and V [..., Hkv, P, D] of the pages `page`, float32 (V only if asked for)."""
    c = s["case"]
    Hkv, P, D = c["Hkv"], c["page"], c["D"]
    views = _pages(c["fmt"], s["pool"], Hkv, P, D)
    v = None
    if c["fmt"] == BF16:
        k = views[0][page].transpose(-2, -3).flatten(-2).flatten(-3, -2).float()
        return k, views[1][page].transpose(-1, -2).flatten(-3, -2).flatten(-3, -2).float() if values else None
    if c["fmt"] == FP8:
        kc, vc, ks, vs = views
        k = _values8(kc[page].transpose(-2, -3).contiguous()).flatten(-2)                    # [.., P/16, 16, D]
        k = (k * torch.exp2(ks[page].float() - 127)[..., None, None]).flatten(-3, -2)
        if values:
            v = _values8(vc[page].movedim(-1, -3).transpose(-1, -2).contiguous()).flatten(-2).flatten(-3, -2)
            v = (v * torch.exp2(vs[page].float() - 127)[..., None, None]).flatten(-3, -2)
        return k, v
    kc, ks, vc, vs = views
    k = s["lut"][kc[page].int()].flatten(-2).transpose(-2, -3).flatten(-4, -3)
    return (k * torch.exp2(ks[page].float() - 127)[..., None]).flatten(-2), None


def _plain_read(s):
    c = s["case"]
    P = c["page"]
    i = torch.arange(s["T"], device="cuda")
    at = s["start"][:, None].long() + i
    live = i < s["count"][:, None]
    page = s["table"].gather(1, torch.where(live, at // P, 0)).clamp(min=0).long()
    k, v = _dense(s, page)                                         # [R, T, Hkv, P, D]
    t = (at % P)[:, :, None, None, None].expand(-1, -1, c["Hkv"], 1, c["D"])
    live = live[:, :, None, None]
    s["k_read"].copy_(torch.where(live, k.gather(3, t)[:, :, :, 0].to(torch.bfloat16), s["k_read"]))
    s["v_read"].copy_(torch.where(live, v.gather(3, t)[:, :, :, 0].to(torch.bfloat16), s["v_read"]))


def _by_head(s, x):
    """[R, pages, Hkv, P, D] -> [R * Hkv, tokens, D]"""
    c = s["case"]
    return x.transpose(1, 2).reshape(c["R"] * c["Hkv"], -1, c["D"])


def _keys(s):
    return _by_head(s, _dense(s, s["table"].clamp(min=0).long(), False)[0])


def _scores(s, k):
    """Scores [R, Hkv, rows, G, tokens] of every row a request can have, -inf where it sees nothing."""
    c = s["case"]
    R, n, Hq, Hkv, D = c["R"], c["gamma"] + 1, c["Hq"], c["Hkv"], c["D"]
    G, S = Hq // Hkv, s["max_pages"] * c["page"]
    i = torch.arange(n, device="cuda")
    live = i <= s["ell"][:, None]
    row = torch.where(live, s["row0"][:, None] + i, 0).long()
    q = s["q"][row].float().view(R, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R * Hkv, n * G, D)
    score = torch.bmm(q, k.transpose(1, 2).contiguous()).mul_(D ** -0.5).view(R, Hkv, n, G, S)
    pos, at = s["length"][:, None] + i, torch.arange(S, device="cuda")
    see = (at <= pos[..., None]) & live[..., None]
    if c["window"]:
        see &= (at > pos[..., None] - c["window"]) | (at < c["sinks"])
    return score.masked_fill_(~see[:, None, :, None], -math.inf)


def _plain_attention(s):
    c = s["case"]
    R, n, Hq, Hkv, D = c["R"], c["gamma"] + 1, c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    k, v = _dense(s, s["table"].clamp(min=0).long())
    score = _scores(s, _by_head(s, k))
    del k
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = score.sum(-1, keepdim=True)
    o = torch.bmm(score.view(R * Hkv, n * G, -1), _by_head(s, v)).view(R, Hkv, n, G, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(R, n, Hq, D)
    lse = (top + torch.log(total))[..., 0].permute(0, 2, 1, 3).reshape(R, n, Hq)
    req, pos = _row_of(s)
    mine = pos - s["length"][req]
    s["out"].copy_(o[req, mine])
    s["lse"].copy_(lse[req, mine])


def _plain_weigh(s):
    c = s["case"]
    R, n, Hkv, G = c["R"], c["gamma"] + 1, c["Hkv"], c["Hq"] // c["Hkv"]
    i = torch.arange(n, device="cuda")
    row = torch.where(i <= s["ell"][:, None], s["row0"][:, None] + i, 0).long()
    lse = s["lse"][row].view(R, n, Hkv, G, 1).transpose(1, 2)
    w = _scores(s, _keys(s)).sub_(lse).exp_().view(R, Hkv * n * G, s["max_pages"], c["page"]).sum((1, 3))
    s["mass"].copy_(torch.where((s["ell"] >= 0)[:, None], 0.75 * s["mass"] + w, s["mass"]))


def _free_bits(ref):
    """One bit per page, set where nobody holds it."""
    bit = torch.ones(1, dtype=torch.int64, device="cuda") << torch.arange(32, device="cuda")
    return ((ref.view(-1, 32) == 0) * bit).sum(-1).to(torch.int32)


def _count(ref, ids, by):
    """Adds `by` to the reference count of every page named in ids (-1: none)."""
    ref.index_add_(0, ids.flatten().clamp(min=0).long(), (ids.flatten() >= 0).to(torch.int32) * by)


def _plain_evict(s):
    c = s["case"]
    P, T, L = c["page"], s["table"], s["length"][:, None]
    col = torch.arange(s["MP"], device="cuda")
    held = (T >= 0) & (col * P < L)
    may = held & ((col + 1) * P <= L - c["recent"]) & (col * P >= c["sinks"])
    over = (held.sum(1) - s["budget"]).clamp(min=0)
    order = torch.argsort(torch.where(may, s["mass"], math.inf), dim=1, stable=True)
    rank = torch.empty_like(order).scatter_(1, order, col.expand_as(order))
    gone = may & (rank < over[:, None])
    _count(s["ref"], torch.where(gone, T, -1), -1)
    T.masked_fill_(gone, -2)  # no page, and evicted
    s["mass"].masked_fill_(gone, 0)
    s["freed"].copy_(gone.sum(1))
    s["bits"].copy_(_free_bits(s["ref"]))


def _plain_history(s):
    """A prompt's tokens: a flag; the tokens kept of the round before: counts."""
    c = s["case"]
    R, V = c["R"], c["V"]
    at = torch.arange(s["prompt"].numel(), device="cuda", dtype=torch.int32)
    req = torch.searchsorted(s["start"], at, right=True) - 1
    flag = torch.zeros(R * V, dtype=torch.int32, device="cuda")
    flag[req * V + s["prompt"]] = -32768
    kept = torch.where(s["ell"] >= 0, torch.minimum(s["n_acc"], s["ell"]) + 1, 0)
    tok = s["x0_before"][:, None] if s["x_before"] is None else torch.cat([s["x0_before"][:, None], s["x_before"]], 1)
    mine = torch.arange(tok.shape[1], device="cuda") < kept[:, None]
    flag.view(R, V).scatter_add_(1, tok.long(), mine.to(torch.int32))
    s["state"].copy_(flag.view(R, V))


def _plain_logits(s):
    c = s["case"]
    V, rows = c["V"], s["rows"]
    row = torch.arange(rows, dtype=torch.int32, device="cuda")
    req = torch.searchsorted(s["row0"], row, right=True) - 1
    mine = row - s["row0"][req]
    # what a row follows: its request's tokens so far, the anchor and the drafts before it
    tok = s["x0"][:, None] if s["x"] is None else torch.cat([s["x0"][:, None], s["x"]], 1)
    state = s["state"].to(torch.int32)
    n = (state & 32767)[req]
    n.scatter_add_(1, tok[req].long(), (torch.arange(tok.shape[1], device="cuda") <= mine[:, None]).to(torch.int32))
    x = s["logits"].float()
    p = s["repetition"][req][:, None]
    x = torch.where((n > 0) | (state < 0)[req], torch.where(x > 0, x / p, x * p), x)
    x -= s["frequency"][req][:, None] * n + s["presence"][req][:, None] * (n > 0)
    if s["bias"] is not None:
        x.scatter_add_(1, s["bias_tok"][req].long(), s["bias"][req])
    if s["mask"] is not None:
        v = torch.arange(V, dtype=torch.int32, device="cuda")
        allowed = s["mask"].repeat_interleave(32, 1)[:, :V].bitwise_right_shift_(v % 32).bitwise_and_(1)
        x.masked_fill_(allowed == 0, -math.inf)
    s["out"].copy_(x)


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    if case["op"] == "evict":
        return None
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "weigh": _exact_attention,
            "logits": _exact_logits}[case["op"]](s)


def _turn(x, w, pos, s):
    """One row of heads [H, D], float64."""
    c, rot = s["case"], s["case"]["rot"]
    x = x.double()
    x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    if rot:
        z = torch.polar(torch.ones_like(s["freq"]), s["freq"] * pos)
        even, odd = (slice(0, rot, 2), slice(1, rot, 2)) if c["adjacent"] else (slice(0, rot // 2), slice(rot // 2, rot))
        y = torch.complex(x[:, even], x[:, odd]) * z
        x[:, even], x[:, odd] = y.real, y.imag
    return x


_E4M3 = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]


def _round8(x):
    """The nearest of the e4m3 values, ties to the even code."""
    v = torch.tensor(_E4M3, dtype=torch.float64, device="cuda")
    y = x.abs()
    i = torch.searchsorted(v, y.contiguous()).clamp(1, 126)
    low, high = y - v[i - 1], v[i] - y
    up = (high < low) | ((high == low) & (i % 2 == 0))
    return v[torch.where(up, i, i - 1)] * torch.sign(x)


def _exact_block(new, codes, byte):
    """A block's values: codes [old tokens, D] with their scale byte and new [n, D], both of one head."""
    e = LOW
    top = float(new.abs().max()) if new.numel() else 0.0
    while top > 448 * 2.0 ** e and e < HIGH:
        e += 1
    old = _values8(codes).double()
    if codes.shape[0]:
        e = max(e, int(byte) - 127)
        old = _round8(old * 2.0 ** (int(byte) - 127 - e))
    return torch.cat([old, _round8(new * 2.0 ** -e)]) * 2.0 ** e


def _exact_append(s):
    c = s["case"]
    Hkv, P, D = c["Hkv"], c["page"], c["D"]
    lens, ells = _lens(c), _ells(c)
    if sum(_up(e + 16, 16) for e in ells if e >= 0) * Hkv > 4000:
        return None
    q, kr, vr = s["q_out"].double(), s["k_read"].double(), s["v_read"].double()
    raw = s["pool"].view(-1, Hkv, 2 * P * D + 16).cpu()
    i = torch.arange(D)
    row = 0
    for r in range(c["R"]):
        n, e = lens[r], ells[r]
        ks, vs = [], []
        for j in range(e + 1):
            q[row] = _turn(s["q"][row], s["wq"], n + j, s)
            ks.append(_turn(s["k"][row], s["wk"], n + j, s))
            vs.append(s["v"][row].double())
            row += 1
        if e < 0:
            continue
        for first in range(n // 16 * 16, n + e + 1, 16):
            a, b = max(first, n), min(first + 16, n + e + 1)
            page, blk = raw[int(s["table"][r, first // P])], first % P // 16
            t = torch.arange(a - first)[:, None]
            for h in range(Hkv):
                at = blk * 16 * D + (i // 16 * 16 + t) * 16 + i % 16
                new = torch.stack([ks[x - n][h] for x in range(a, b)])
                z = _exact_block(new, page[h][at].cuda(), page[h][2 * P * D + blk])
                kr[r, first - n // 16 * 16:b - n // 16 * 16, h] = z
                at = P * D + blk * 16 * D + ((t // 8 * 32 + i % 32) * (D // 32) + i // 32) * 8 + t % 8
                new = torch.stack([vs[x - n][h] for x in range(a, b)])
                z = _exact_block(new, page[h][at].cuda(), page[h][2 * P * D + 8 + blk])
                vr[r, first - n // 16 * 16:b - n // 16 * 16, h] = z
    return {"q": q, "k": kr, "v": vr}


def _exact_attention(s):
    """Attention's outputs, or the weights of the pages from the log-sums as given."""
    c = s["case"]
    Hq, Hkv, D, P, weigh = c["Hq"], c["Hkv"], c["D"], c["page"], c["op"] == "weigh"
    lens, ells = _lens(c), _ells(c)
    if sum(n * (e + 1) for n, e in zip(lens, ells)) * Hq * D > 3e11:
        return None
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    e4m3 = torch.tensor(_E4M3 + [math.nan], dtype=torch.float64, device="cuda")
    e4m3 = torch.cat([e4m3, -e4m3])
    lse = s["lse"].double()
    out = s["first"].double() if weigh else s["out"].double()
    row = 0
    for r in range(c["R"]):
        n = ells[r] + 1
        if n == 0:
            continue
        N = lens[r] + n
        x = s["pool"][s["table"][r, :_up(N, P)].long()]
        v = None
        if c["fmt"] == BF16:
            x = x.view(torch.bfloat16).view(-1, Hkv, 2, P // 16, 16 * D)
            k = x[:, :, 0].reshape(-1, Hkv, P // 16, D // 8, 16, 8).permute(1, 0, 2, 4, 3, 5).reshape(Hkv, -1, D).double()
        elif c["fmt"] == FP8:
            x = x.view(x.shape[0], Hkv, -1)
            a, b = P * D, P // 16
            k = e4m3[x[:, :, :a].int()].reshape(-1, Hkv, b, D // 16, 16, 16).permute(1, 0, 2, 4, 3, 5)
            k = k * torch.exp2(x[:, :, 2 * a:2 * a + b].double() - 127).transpose(0, 1)[..., None, None, None]
            v = e4m3[x[:, :, a:2 * a].int()].reshape(-1, Hkv, b, 2, 32, D // 32, 8).permute(1, 0, 2, 3, 6, 5, 4)
            v = v * torch.exp2(x[:, :, 2 * a + 8:2 * a + 8 + b].double() - 127).transpose(0, 1)[..., None, None, None, None]
            k, v = k.reshape(Hkv, -1, D), v.reshape(Hkv, -1, D)[:, :N]
        else:
            x = x.view(x.shape[0], Hkv, -1)
            a, b = P * D // 2, P * D // 32
            k = x[:, :, :a].reshape(-1, Hkv, P // 16, D // 32, 16, 16).permute(1, 0, 2, 4, 3, 5).reshape(Hkv, -1, D // 2)
            k = torch.stack([lut[(k & 15).int()], lut[(k >> 4).int()]], -1).view(Hkv, -1, D // 32, 32)
            sc = x[:, :, a:a + b].reshape(-1, Hkv, P, D // 32).transpose(0, 1).reshape(Hkv, -1, D // 32, 1)
            k = (k * torch.exp2(sc.double() - 127)).view(Hkv, -1, D)
        q = s["q"][row:row + n].double().view(n, Hkv, Hq // Hkv, D).permute(1, 0, 2, 3).reshape(Hkv, -1, D)
        score = torch.bmm(q, k[:, :N].transpose(1, 2).contiguous()).view(Hkv, n, Hq // Hkv, N) / math.sqrt(D)
        for i in range(n):
            p = lens[r] + i
            score[:, i, :, p + 1:] = -math.inf
            if c["window"]:
                score[:, i, :, min(c["sinks"], p):max(0, p - c["window"] + 1)] = -math.inf
        if weigh:
            w = torch.exp(score - lse[row:row + n].view(n, Hkv, -1).transpose(0, 1)[..., None]).sum((0, 1, 2))
            out[r] *= 0.75
            out[r].index_add_(0, torch.arange(N, device="cuda") // P, w)
        else:
            z = torch.logsumexp(score, -1)
            o = torch.bmm(torch.exp(score - z[..., None]).view(Hkv, -1, N), v.contiguous())
            out[row:row + n] = o.view(Hkv, n, Hq // Hkv, D).permute(1, 0, 2, 3).reshape(n, Hq, D)
            lse[row:row + n] = z.permute(1, 0, 2).reshape(n, Hq)
        row += n
    return {"mass": out} if weigh else {"out": out, "lse": lse}


def _exact_logits(s):
    c = s["case"]
    V, lens, ells = c["V"], _lens(c), _ells(c)
    out = s["logits"].double()
    row = 0
    for r in range(c["R"]):
        if c["fresh"]:
            at = int(s["start"][r])
            prompt = torch.bincount(s["prompt"][at:at + lens[r]], minlength=V) > 0
            kept = [] if ells[r] < 0 else [s["x0_before"][r:r + 1]]
            if ells[r] >= 0 and c["gamma"]:
                kept.append(s["x_before"][r, :min(int(s["n_acc"][r]), ells[r])])
            n = torch.bincount(torch.cat(kept), minlength=V) if kept else torch.zeros(V, dtype=torch.int64, device="cuda")
        else:
            n = s["state"][r].long()
            prompt = n < 0
            n = torch.where(prompt, n + 32768, n)
        rep, pres, freq = (float(s[k][r]) for k in ("repetition", "presence", "frequency"))
        for i in range(ells[r] + 1):
            n[s["x0"][r] if i == 0 else s["x"][r, i - 1]] += 1
            x = out[row]
            hit = prompt | (n > 0)
            x = torch.where(hit, torch.where(x > 0, x / rep, x * rep), x) - freq * n - pres * (n > 0)
            if s["bias"] is not None:
                x[s["bias_tok"][r].long()] += s["bias"][r].double()
            if s["mask"] is not None:
                bits = (s["mask"][row].long() & 0xFFFFFFFF)[:, None] >> torch.arange(32, device="cuda") & 1
                x[bits.flatten()[:V] == 0] = -math.inf
            out[row] = x
            row += 1
    return {"out": out, "state": None} if c["fresh"] else {"out": out}
