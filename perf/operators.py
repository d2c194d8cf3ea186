"""The paged-cache operators of a verification round, as measured cases.

A round drafts a block per request, admits ell[r] drafts of request r and
verifies them in one flattened batch: rows row0[r] .. row0[r] + ell[r] of the
target's forward pass, at positions len[r] .. len[r] + ell[r] of the request's
cache.  The operators here are what that forward pass and its roll-back do to
a paged key/value cache:

  append     norms of queries and keys per head and the position rotation in
             one pass; keys and values go to the pages (16 or 4 bits)
  attention  the rows' attention over the pages: causal, grouped heads, an
             optional sliding window with the first tokens still visible;
             over 16-bit pages and over 4-bit pages
  pages      reserve / copy-on-write / commit / fork / compact / copy

Every operator has a plain form (elementary torch, float32, float64 where a
4-bit rounding border or a far position's angle needs it) and the framework's
call; `exact` computes the same from the definition in float64.

Page layouts (what the plain forms index): a page holds P tokens of every
key/value head.  16-bit: [head][K, V][P/16] blocks of 16 tokens, a K block
[D/8][16 tokens][8 dims], a V block [2][D][8 tokens].  4-bit: per head K codes
[P/16][D/32][16 tokens][16 bytes], K scale bytes [P][D/32] (value 2^(b-127)),
V codes [P/16][2][32 dims][D/32][4 bytes = 8 tokens], V scales [P] float32;
a code is sign and magnitude of {0, 0.5, 1, 1.5, 2, 3, 4, 6}.
"""

import math

import torch

own = False

EPS = 1e-6
BF16, FP4 = 1, 2


# ------------------------------------------------------------------ cases

def _attn(name, fmt, R, gamma, Hq, Hkv, D, page, ctx, window=0, sinks=0, ell="ragged"):
    return dict(name=name, op="attention", fmt=fmt, R=R, gamma=gamma, Hq=Hq, Hkv=Hkv, D=D, page=page, ctx=ctx,
                window=window, sinks=sinks, ell=ell)


def _app(name, fmt, R, gamma, Hq, Hkv, D, page, ctx, rot, adjacent=False, packed=False, ell="ragged"):
    return dict(name=name, op="append", fmt=fmt, R=R, gamma=gamma, Hq=Hq, Hkv=Hkv, D=D, page=page, ctx=ctx, rot=rot,
                adjacent=adjacent, packed=packed, ell=ell)


def listed():
    return [
        # one request, one token: what every decode step of a lone user waits for
        _app("append_r1_token", BF16, 1, 0, 32, 8, 128, 64, 1000, 128, ell="full"),
        # the batched round (128 requests, up to 17 rows each, 7168 wide: 56 heads), fused projection rows
        _app("append_r128_g16_packed", BF16, 128, 16, 56, 8, 128, 64, 250, 128, packed=True),
        # 32 requests at their full block into 4-bit pages, and those rows read back
        _app("append_fp4_r32_g16", FP4, 32, 16, 32, 8, 128, 32, 500, 128, ell="full"),
        # prompts entering the cache in chunks of 512 rows, half of each head rotated, adjacent pairs
        _app("append_prompt_r4_g511", BF16, 4, 511, 32, 8, 128, 64, 1500, 64, adjacent=True, ell="full"),
        # one request, one token, a short odd context: latency
        _attn("attn_r1_token_1023", BF16, 1, 0, 32, 8, 128, 64, 1023, ell="full"),
        # the batched round over ragged contexts up to 8192, nothing hidden
        _attn("attn_r128_g16_8192", BF16, 128, 16, 56, 8, 128, 64, 8192),
        # a window of 1024 and 4 first tokens, small pages, 32 requests at their full block
        _attn("attn_window_r32_g16", BF16, 32, 16, 32, 8, 128, 16, 6000, window=1024, sinks=4, ell="full"),
        # one request with a long odd context: the split over a long axis
        _attn("attn_r1_g16_131055", BF16, 1, 16, 32, 8, 128, 64, 131055, ell="full"),
        # one token each for 32 requests over 4-bit pages
        _attn("attn_fp4_r32_token_16384", FP4, 32, 0, 32, 8, 128, 64, 16384, ell="full"),
        # the batched round over 4-bit pages, contexts up to 16384
        _attn("attn_fp4_r128_g16_16384", FP4, 128, 16, 56, 8, 128, 64, 16384),
        # a round's bookkeeping: beams forked, pages reserved and copied where shared, commit after verification
        dict(name="pages_round_r128", op="round", R=128, gamma=16, Hkv=8, D=128, page=16, ctx=250, spare=256, layers=1,
             window=0, sinks=0),
        # a fragmented pool drawn together: 2 layers, 256 KB pages
        dict(name="pages_compact_2048", op="compact", R=64, Hkv=8, D=128, page=64, ctx=1200, n_pages=2048, layers=2),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["append", "append", "attention", "attention", "attention", "round", "compact"])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 7, 8])
    D = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    if op == "round":
        return dict(op=op, R=_log(rng, 1, 160), gamma=rng.randint(0, 16), Hkv=Hkv, D=D, page=page,
                    ctx=_log(rng, 20, 300), spare=rng.randint(0, 300), layers=rng.choice([1, 2]),
                    window=rng.choice([0, 0, 50]), sinks=rng.choice([0, 4, 33]))
    if op == "compact":
        return dict(op=op, R=_log(rng, 1, 64), Hkv=Hkv, D=D, page=page, ctx=_log(rng, 100, 1200),
                    n_pages=_log(rng, 300, min(2000, 250_000_000 // (Hkv * page * D * 4))), layers=rng.choice([1, 2]))
    fmt = rng.choice([BF16, FP4])
    R = _log(rng, 1, 128)
    gamma = rng.choice([0, 0, rng.randint(1, 16), rng.randint(1, 64), 16])
    ell = rng.choice(["ragged", "full"])
    if op == "append":
        rot = rng.choice([0, D // 2, D, D])
        return _app(None, fmt, R, gamma, Hq, Hkv, D, page, _log(rng, 1, 300), rot, rng.choice([False, True]),
                    rng.choice([False, True]), ell)
    # a drawn attention stays under the largest listed one: its cache by the tokens it may hold, its
    # products by the rows of a full block
    most = 800_000 * 8 * 128 // (Hkv * D)
    ctx = _log(rng, 1, max(8, min(60_000, most // R, 400_000_000 // (R * (gamma + 1) * Hq))))
    window = rng.choice([0, 0, _log(rng, 1, 4096)])
    return _attn(None, fmt, R, gamma, Hq, Hkv, D, page, ctx, window, rng.choice([0, 4, 64]) if window else 0, ell)


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


def _token_bytes(fmt, D):
    """Bytes of one token of one key/value head."""
    return 4 * D if fmt == BF16 else D + D // 32 + 4


def work(case):
    op = case["op"]
    if op in ("append", "attention"):
        lens, ells = _lens(case), _ells(case)
        rows = sum(e + 1 for e in ells)
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        tb = _token_bytes(case["fmt"], D)
        if op == "append":
            b = rows * (Hq + 2 * Hkv) * D * 2 + rows * Hq * D * 2 + rows * Hkv * tb
            if case["fmt"] == FP4:
                b += rows * Hkv * (tb + 4 * D)
            return {"bytes": b, "flops": rows * (Hq + Hkv) * D * 8}
        W, S = case["window"], case["sinks"]
        tokens = seen = 0
        for n, e in zip(lens, ells):
            if e < 0:
                continue
            for i in range(e + 1):
                p = n + i
                low = max(0, p - W + 1) if W else 0
                seen += p + 1 - low + min(S, low)
            low = max(0, n - W + 1) if W else 0
            tokens += n + e + 1 - low + min(S, low)
        return {"bytes": tokens * Hkv * tb + rows * Hq * (4 * D + 4), "flops": 4 * seen * Hq * D}
    pb = case["Hkv"] * case["page"] * _token_bytes(BF16, case["D"])
    s = _page_shapes(case)
    if op == "round":
        tab = case["R"] * s["max_pages"] * 4
        return {"bytes": 2 * s["copies"] * pb * case["layers"] + 4 * tab + 8 * s["n_pages"], "flops": 0}
    return {"bytes": 2 * s["copies"] * pb * case["layers"] + 2 * case["R"] * s["max_pages"] * 4 + 12 * s["n_pages"],
            "flops": 0}


def _parents(case):
    """Every eighth slot is forked from its left neighbour, every sixteenth let go."""
    return [(-1 if r % 16 == 9 else r - 1 if r % 8 == 4 else r) for r in range(case["R"])]


def _page_shapes(case):
    """Sizes of the page cases, and how many pages they copy."""
    R, P, lens = case["R"], case["page"], _lens(case)
    if case["op"] == "round":
        max_pages = _up(case["ctx"] + case["gamma"] + 1, P) + 1
        used = sum(_up(n, P) for n in lens)
        n_pages = _up(used + case["spare"] + 32, 32) * 32
        par = _parents(case)
        return dict(max_pages=max_pages, n_pages=n_pages, copies=sum(p >= 0 and p != r and lens[p] % P > 0 for r, p in enumerate(par)))
    max_pages = _up(case["ctx"], P)
    held = min(sum(_up(n, P) for n in lens), case["n_pages"])
    n_pages = _up(case["n_pages"], 32) * 32
    return dict(max_pages=max_pages, n_pages=n_pages, copies=int(held * (1 - held / n_pages)))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _code_bytes(n, g):
    """Random pairs of 4-bit codes, as often as a quantised normal variable takes them."""
    out = torch.empty(n, dtype=torch.uint8, device="cuda")
    for a in range(0, n, 1 << 26):
        m = min(1 << 26, n - a)
        x = torch.randn(2 * m, generator=g, device="cuda", dtype=torch.float16) * 2.3
        y = x.abs()
        c = torch.zeros(2 * m, dtype=torch.uint8, device="cuda")
        for t in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
            c += y > t
        c += (x < 0).to(torch.uint8) * 8
        c = c.view(m, 2)
        out[a:a + m] = c[:, 0] + c[:, 1] * 16
    return out


def _pool(fmt, n_pages, Hkv, D, P, g):
    """A pool that earlier rounds filled."""
    if fmt == BF16:
        pool = torch.empty(n_pages * Hkv * 2 * P * D, dtype=torch.bfloat16, device="cuda")
        for a in range(0, pool.numel(), 1 << 28):
            pool[a:a + (1 << 28)].normal_(generator=g)
        return pool.view(torch.uint8).view(n_pages, -1)
    hb = P * _token_bytes(FP4, D)
    pool = _code_bytes(n_pages * Hkv * hb, g).view(n_pages, Hkv, hb)
    a = P * D // 2
    pool[:, :, a:a + P * D // 32] = torch.randint(124, 127, (n_pages, Hkv, P * D // 32), generator=g, device="cuda",
                                                  dtype=torch.uint8)
    s = torch.rand(n_pages, Hkv, P, generator=g, device="cuda") * 0.3 + 0.3
    pool[:, :, 2 * a + P * D // 32:] = s.view(torch.uint8).view(n_pages, Hkv, 4 * P)
    return pool.view(n_pages, -1)


def _tables(case, need, max_pages, n_pages, g):
    """Pages in no order: request r holds need[r] of them."""
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(need), max_pages), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += n
    return table


def prepare(case, seed):
    g = _gen(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    op = case["op"]
    if op in ("round", "compact"):
        return _prepare_pages(case, g)
    R, gamma, Hq, Hkv, D, P = (case[k] for k in ("R", "gamma", "Hq", "Hkv", "D", "page"))
    lens, ells = _lens(case), _ells(case)
    need = [_up(n + e + 1, P) for n, e in zip(lens, ells)]
    max_pages = _up(case["ctx"] + gamma + 1, P)
    n_pages = sum(need) + 5
    row0, rows = [], 0
    for e in ells:
        row0.append(rows)
        rows += e + 1
    v16 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    s = dict(case=case, rows=rows, lut=torch.stack([v16.repeat(16), v16.repeat_interleave(16)], -1), max_pages=max_pages, length=torch.tensor(lens, **i32), ell=torch.tensor(ells, **i32),
             row0=torch.tensor(row0, **i32), table=_tables(case, need, max_pages, n_pages, g),
             pool=_pool(case["fmt"], n_pages, Hkv, D, P, g))
    bf = dict(dtype=torch.bfloat16, device="cuda")
    if op == "attention":
        s["q"] = (1.5 * torch.randn(rows, Hq, D, generator=g, device="cuda")).to(torch.bfloat16)
        s["out"] = torch.zeros(rows, Hq, D, **bf)
        s["lse"] = torch.zeros(rows, Hq, dtype=torch.float32, device="cuda")
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
    if case["fmt"] == FP4:
        s["k_read"] = torch.zeros(R, gamma + 1, Hkv, D, **bf)
        s["v_read"] = torch.zeros(R, gamma + 1, Hkv, D, **bf)
        s["count"] = s["ell"] + 1
    return s


def _prepare_pages(case, g):
    i32 = dict(dtype=torch.int32, device="cuda")
    R, P, Hkv, D = case["R"], case["page"], case["Hkv"], case["D"]
    sh, lens = _page_shapes(case), _lens(case)
    MP, N = sh["max_pages"], sh["n_pages"]
    need, left = [], N
    for n in lens:  # a compact case's pool may be smaller than its requests would fill
        need.append(min(_up(n, P), left))
        left -= need[-1]
    lens = [min(n, k * P) for n, k in zip(lens, need)]
    words = N // 32
    # one buffer holds the whole bookkeeping, so that a pass starts from the same state with one copy
    first = torch.zeros(R * MP + R + N + words, **i32)
    s = dict(case=case, P=P, MP=MP, N=N, first=first, state=torch.zeros_like(first))
    table = _tables(case, need, MP, N, g)
    ref = torch.zeros(N, **i32)
    ref[table[table >= 0].long()] = 1
    first[:R * MP] = table.flatten()
    first[R * MP:R * MP + R] = torch.tensor(lens, **i32)
    first[R * MP + R:R * MP + R + N] = ref
    first[R * MP + R + N:] = _free_bits(ref)
    st = s["state"]
    s["table"] = st[:R * MP].view(R, MP)
    s["length"] = st[R * MP:R * MP + R]
    s["ref"] = st[R * MP + R:R * MP + R + N]
    s["bits"] = st[R * MP + R + N:]
    held = int((ref > 0).sum())
    s["most"] = R if case["op"] == "round" else min(held, N - held)  # pairs that a pass can have
    s["pairs"] = torch.zeros(R if case["op"] == "round" else N // 2, 2, **i32)
    s["n_pairs"] = torch.zeros(1, **i32)
    s["pool"] = torch.stack([_pool(BF16, N, Hkv, D, P, g) for _ in range(case["layers"])])
    if case["op"] == "round":
        ell = [int((case["gamma"] + 1) * ((r * 0.7548776662466927 + 0.31) % 1.0) ** 2) for r in range(R)]
        s["ell"] = torch.tensor(ell, **i32)
        s["n_acc"] = torch.tensor([int((e + 1) * ((r * 0.5698402909980532) % 1.0)) for r, e in enumerate(ell)], **i32)
        s["parent"] = torch.tensor(_parents(case), **i32)
        s["ell_out"] = torch.zeros(R, **i32)
        s["status"] = torch.zeros(1, **i32)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if op == "append":
        return _run_append(s)
    if op == "attention":
        return _run_attention(s)
    return _run_round(s) if op == "round" else _run_compact(s)


def _run_append(s):
    c = s["case"]
    if own:
        from semi_ar_draft_round_amd import binding as B
        B.dspark_cache_append(s["q"], s["k"], s["v"], s["pool"], s["table"], s["length"], s["ell"], c["gamma"],
                              fmt=c["fmt"], page=c["page"], wq=s["wq"], wk=s["wk"], eps=EPS, freq=s["freq"],
                              adjacent=c["adjacent"], row0=s["row0"], q_out=s["q_out"])
        if c["fmt"] == FP4:
            B.dspark_cache_read(s["pool"], s["table"], s["length"], s["count"], c["gamma"] + 1, fmt=c["fmt"],
                                page=c["page"], heads_kv=c["Hkv"], dim=c["D"], k=s["k_read"], v=s["v_read"])
    else:
        _plain_append(s)
        if c["fmt"] == FP4:
            _plain_read(s)
    if c["fmt"] == FP4:
        return {"q": s["q_out"], "k": s["k_read"], "v": s["v_read"]}
    return {"q": s["q_out"], "pool": s["pool"].view(torch.bfloat16)}


def _run_attention(s):
    c = s["case"]
    if own:
        from semi_ar_draft_round_amd import binding as B
        B.dspark_cache_attention(s["q"], s["pool"], s["table"], s["length"], s["ell"], c["gamma"], fmt=c["fmt"],
                                 page=c["page"], heads_kv=c["Hkv"], window=c["window"], sinks=c["sinks"],
                                 row0=s["row0"], out=s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    return _plain_attention(s)


def _state_out(s):
    return {"table": s["table"], "length": s["length"], "ref": s["ref"], "bits": s["bits"], "n_pairs": s["n_pairs"],
            "pool": s["pool"]}


def _run_round(s):
    c = s["case"]
    s["state"].copy_(s["first"])
    if own:
        from semi_ar_draft_round_amd import binding as B
        B.dspark_cache_fork(s["table"], s["length"], s["ref"], s["bits"], s["parent"], page=c["page"])
        B.dspark_cache_reserve(s["table"], s["length"], s["ref"], s["bits"], s["ell"], c["gamma"], page=c["page"],
                               ell_out=s["ell_out"], pairs=s["pairs"], n_pairs=s["n_pairs"], status=s["status"])
        B.dspark_cache_copy(s["pool"], s["pairs"], s["n_pairs"])
        B.dspark_cache_commit(s["table"], s["length"], s["ref"], s["bits"], s["ell_out"], s["n_acc"], c["gamma"],
                              page=c["page"], window=c["window"], sinks=c["sinks"])
    else:
        _plain_fork(s)
        _plain_reserve(s)
        _plain_copy(s)
        _plain_commit(s)
    return _state_out(s) | {"ell": s["ell_out"], "status": s["status"]}


def _run_compact(s):
    s["state"].copy_(s["first"])
    if own:
        from semi_ar_draft_round_amd import binding as B
        B.dspark_cache_compact(s["table"], s["ref"], s["bits"], pairs=s["pairs"], n_pairs=s["n_pairs"])
        B.dspark_cache_copy(s["pool"], s["pairs"], s["n_pairs"])
    else:
        _plain_compact(s)
        _plain_copy(s)
    return _state_out(s)


# ------------------------------------------------------------------ plain forms

def _pages16(pool, Hkv, P, D):
    """K [n, Hkv, P/16, D/8, 16, 8] and V [n, Hkv, P/16, 2, D, 8] of 16-bit pages, as views."""
    x = pool.view(torch.bfloat16).view(-1, Hkv, 2, P // 16, 16 * D)
    return x[:, :, 0].unflatten(-1, (D // 8, 16, 8)), x[:, :, 1].unflatten(-1, (2, D, 8))


def _pages4(pool, Hkv, P, D):
    """K codes, K scales, V codes and V scales of 4-bit pages, as views."""
    x = pool.view(pool.shape[0], Hkv, -1)
    a, b = P * D // 2, P * D // 2 + P * D // 32
    return (x[:, :, :a].unflatten(-1, (P // 16, D // 32, 16, 16)), x[:, :, a:b].unflatten(-1, (P, D // 32)),
            x[:, :, b:b + a].unflatten(-1, (P // 16, 2, 32, D // 32, 4)), x[:, :, b + a:].view(torch.float32))


def _code(x, one=1.0):
    """e2m1 codes of x / one, nearest, ties to the even code.  The borders are multiples of `one`, so that
    16-bit x and one are compared exactly."""
    y = x.abs()
    c = ((y > 0.25 * one).to(torch.uint8) + (y >= 0.75 * one) + (y > 1.25 * one) + (y >= 1.75 * one) + (y > 2.5 * one)
         + (y >= 3.5 * one) + (y > 5.0 * one))
    return c + (x < 0).to(torch.uint8) * 8


def _value(codes, pairs):
    """The float32 values of bytes that hold two codes each (`pairs`: both values of every byte): the last
    axis doubles, low nibble first."""
    return pairs[codes.int()].flatten(-2)


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


def _plain_append(s):
    c = s["case"]
    Hkv, P, D = c["Hkv"], c["page"], c["D"]
    req, pos = _row_of(s)
    s["q_out"].copy_(_norm_rotate(s["q"], s["wq"], pos, s, torch.float32))
    page, t = s["table"][req, pos // P].long(), pos % P
    blk, tt = t // 16, t % 16
    if c["fmt"] == BF16:
        k = _norm_rotate(s["k"], s["wk"], pos, s, torch.float32).to(torch.bfloat16)
        kp, vp = _pages16(s["pool"], Hkv, P, D)
        kp[page, :, blk, :, tt] = k.unflatten(-1, (D // 8, 8))
        vp[page, :, blk, tt // 8, :, tt % 8] = s["v"]
        return
    k = _norm_rotate(s["k"], s["wk"], pos, s, torch.float64).unflatten(-1, (D // 32, 32))
    kc, ks, vc, vs = _pages4(s["pool"], Hkv, P, D)
    top = k.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(top))
    e = torch.where(torch.exp2(e) > top, e - 1, torch.where(torch.exp2(e + 1) <= top, e + 1, e)) - 2
    e = torch.where(top * torch.exp2(-e) > 7, e + 1, e).clamp(-126, 127)
    code = _code(k * torch.exp2(-e))
    kc[page, :, blk, :, tt] = code[..., 0::2] + code[..., 1::2] * 16
    ks[page, :, t] = (e[..., 0] + 127).to(torch.uint8)
    v = s["v"].float()
    top = v.abs().amax(-1, keepdim=True)
    scale = top[..., 0] / 6
    code = torch.where(top > 0, _code(6 * v, top), 0)
    # token tt's nibble of the 4-byte word that holds 8 tokens of one dim; dim d is [d % 32][d // 32]
    code = code.unflatten(-1, (D // 32, 32)).transpose(-1, -2)
    vs[page, :, t] = scale
    # two tokens share a byte: rows that are neighbours in it both write the whole byte, the same one
    byte, odd = tt % 8 // 2, (tt % 2 == 1)[:, None, None, None]
    word = vc[page, :, blk, tt // 8, :, :, byte]
    pair = (req[1:] == req[:-1]) & (pos[1:] == pos[:-1] + 1)
    no = torch.zeros_like(pair[:1]) if pair.numel() else torch.zeros(1, dtype=torch.bool, device="cuda")
    has_next, has_prev = (x[:, None, None, None] for x in (torch.cat([pair, no]), torch.cat([no, pair])))
    low = torch.where(odd, torch.where(has_prev, code.roll(1, 0), word & 15), code)
    high = torch.where(odd, code, torch.where(has_next, code.roll(-1, 0), word >> 4))
    vc[page, :, blk, tt // 8, :, :, byte] = low + high * 16


def _dense(s, page):
    """K and V [..., Hkv, P, D] of the pages `page`, float32."""
    c = s["case"]
    Hkv, P, D = c["Hkv"], c["page"], c["D"]
    if c["fmt"] == BF16:
        kp, vp = _pages16(s["pool"], Hkv, P, D)
        k = kp[page].transpose(-2, -3).flatten(-2)                 # [.., Hkv, P/16, 16, D]
        v = vp[page].transpose(-1, -2).flatten(-3, -2)             # [.., Hkv, P/16, 16, D]
        return k.flatten(-3, -2).float(), v.flatten(-3, -2).float()
    kc, ks, vc, vs = _pages4(s["pool"], Hkv, P, D)
    k = _value(kc[page], s["lut"]).transpose(-2, -3).flatten(-4, -3)         # [.., Hkv, P, D/32, 32]
    k = (k * torch.exp2(ks[page].float() - 127)[..., None]).flatten(-2)
    v = _value(vc[page], s["lut"])                                           # [.., P/16, 2, 32, D/32, 8 tokens]
    v = v.movedim(-1, -3).transpose(-1, -2).flatten(-2).flatten(-4, -2)
    return k, v * vs[page][..., None]


def _plain_read(s):
    c = s["case"]
    P, T = c["page"], c["gamma"] + 1
    at = s["length"][:, None].long() + torch.arange(T, device="cuda")
    live = torch.arange(T, device="cuda") < s["count"][:, None]
    page = s["table"].gather(1, torch.where(live, at // P, 0)).clamp(min=0).long()
    k, v = _dense(s, page)                                         # [R, T, Hkv, P, D]
    t = (at % P)[:, :, None, None, None].expand(-1, -1, c["Hkv"], 1, c["D"])
    live = live[:, :, None, None]
    s["k_read"].copy_(torch.where(live, k.gather(3, t)[:, :, :, 0].to(torch.bfloat16), s["k_read"]))
    s["v_read"].copy_(torch.where(live, v.gather(3, t)[:, :, :, 0].to(torch.bfloat16), s["v_read"]))


def _plain_attention(s):
    c = s["case"]
    R, n, Hq, Hkv, D, P = c["R"], c["gamma"] + 1, c["Hq"], c["Hkv"], c["D"], c["page"]
    G, S = Hq // Hkv, s["max_pages"] * P
    k, v = _dense(s, s["table"].clamp(min=0).long())               # [R, pages, Hkv, P, D]
    k, v = (x.transpose(1, 2).reshape(R * Hkv, S, D) for x in (k, v))
    i = torch.arange(n, device="cuda")
    live = i <= s["ell"][:, None]
    row = torch.where(live, s["row0"][:, None] + i, 0).long()
    q = s["q"][row].float().view(R, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R * Hkv, n * G, D)
    score = torch.bmm(q, k.transpose(1, 2).contiguous()).mul_(D ** -0.5).view(R, Hkv, n, G, S)
    pos, at = s["length"][:, None] + i, torch.arange(S, device="cuda")
    see = (at <= pos[..., None]) & live[..., None]
    if c["window"]:
        see &= (at > pos[..., None] - c["window"]) | (at < c["sinks"])
    score.masked_fill_(~see[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = score.sum(-1, keepdim=True)
    o = torch.bmm(score.view(R * Hkv, n * G, S), v).view(R, Hkv, n, G, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(R, n, Hq, D)
    lse = (top + torch.log(total))[..., 0].permute(0, 2, 1, 3).reshape(R, n, Hq)
    req, pos = _row_of(s)
    mine = pos - s["length"][req]
    s["out"].copy_(o[req, mine])
    s["lse"].copy_(lse[req, mine])
    return {"out": s["out"], "lse": s["lse"]}


def _free_bits(ref):
    """One bit per page, set where nobody holds it."""
    bit = torch.ones(1, dtype=torch.int64, device="cuda") << torch.arange(32, device="cuda")
    return ((ref.view(-1, 32) == 0) * bit).sum(-1).to(torch.int32)


def _count(ref, ids, by):
    """Adds `by` to the reference count of every page named in ids (-1: none)."""
    ref.index_add_(0, ids.flatten().clamp(min=0).long(), (ids.flatten() >= 0).to(torch.int32) * by)


def _plain_fork(s):
    T, L, ref, par, P = s["table"], s["length"], s["ref"], s["parent"], s["P"]
    R = T.shape[0]
    ar, col = torch.arange(R, device="cuda"), torch.arange(s["MP"], device="cuda")
    keep = ((par == ar) | (par >= R) | (par < -1))[:, None]
    src = par.clamp(0, R - 1).long()
    some = (par >= 0)[:, None] & (col < ((L[src] + P - 1) // P)[:, None])
    new = torch.where(some, T[src], -1)
    _count(ref, torch.where(keep, -1, new), 1)
    _count(ref, torch.where(keep, -1, T), -1)
    L.copy_(torch.where(keep[:, 0], L, torch.where(par >= 0, L[src], 0)))
    T.copy_(torch.where(keep, T, new))
    s["bits"].copy_(_free_bits(ref))


def _plain_reserve(s):
    T, L, ref, P, MP = s["table"], s["length"], s["ref"], s["P"], s["MP"]
    R, gamma = T.shape[0], s["case"]["gamma"]
    ar, col = torch.arange(R, device="cuda"), torch.arange(MP, device="cuda")
    n = s["ell"].clamp(-1, gamma) + 1
    p0, p1 = L // P, (L + n + P - 1) // P
    act = (n > 0) & (p1 <= MP)
    tail = T[ar, p0.clamp(max=MP - 1).long()]
    tref = ref[tail.clamp(min=0).long()]
    sh = act & (L % P != 0) & (tail >= 0)
    before = ((tail[:, None] == tail) & sh[:, None] & sh).tril(-1).sum(1)
    copy = sh & (tref - before > 1)
    exempt = sh & ~copy & (tref > 1)
    need = act[:, None] & (col >= p0[:, None]) & (col < p1[:, None]) & (T < 0)
    cnt = need.sum(1) + copy
    total = cnt.cumsum(0)
    free = (ref == 0).sum()
    ok = act & torch.where(cnt > 0, total <= free, ~exempt | (total - cnt <= free)) & (~exempt | (total - cnt <= free))
    ids = torch.argsort((ref > 0).to(torch.int8), stable=True).to(torch.int32)
    base = (total - cnt)[:, None]
    rank = (base + copy[:, None] + need.cumsum(1) - 1).clamp(0, s["N"] - 1)
    copy &= ok
    fresh = torch.where(copy, ids[base[:, 0].clamp(max=s["N"] - 1)], -1)
    new = torch.where(need & ok[:, None], ids[rank], -1)
    _count(ref, torch.where(copy, tail, -1), -1)
    _count(ref, fresh, 1)
    _count(ref, new, 1)
    T.copy_(torch.where(new >= 0, new, torch.where(copy[:, None] & (col == p0[:, None]), fresh[:, None], T)))
    order = torch.argsort((~copy).to(torch.int8), stable=True)
    s["pairs"][:R] = torch.stack([tail[order], fresh[order]], 1)
    s["n_pairs"].copy_(copy.sum().view(1))
    s["ell_out"].copy_(torch.where(ok, n - 1, -1))
    s["status"].copy_((((n > 0) & ~ok).any() * 7).view(1))
    s["bits"].copy_(_free_bits(ref))


def _plain_commit(s):
    T, L, ref, P, c = s["table"], s["length"], s["ref"], s["P"], s["case"]
    col = torch.arange(s["MP"], device="cuda")
    ell = s["ell_out"]
    act = (ell >= 0)[:, None]
    L.copy_(torch.where(act[:, 0], (L + torch.minimum(s["n_acc"].clamp(min=0), ell) + 1).clamp(max=s["MP"] * P), L))
    gone = col >= ((L + P - 1) // P)[:, None]
    if c["window"]:
        gone |= ((col + 1) * P <= (L - c["window"] + 1)[:, None]) & (col * P >= c["sinks"])
    gone &= act & (T >= 0)
    _count(ref, torch.where(gone, T, -1), -1)
    T.masked_fill_(gone, -1)
    s["bits"].copy_(_free_bits(ref))


def _plain_compact(s):
    T, ref, N = s["table"], s["ref"], s["N"]
    ids = torch.arange(N, device="cuda")
    used = ref > 0
    U = used.sum()
    out, hole = used & (ids >= U), ~used & (ids < U)
    src, dst = torch.argsort((~out).to(torch.int8), stable=True), torch.argsort((~hole).to(torch.int8), stable=True)
    n = out.sum()
    to = torch.empty_like(ids)
    to[src] = torch.where(ids < n, dst, src)
    moved = torch.zeros_like(ref).index_add_(0, to, ref)
    ref.copy_(moved)
    T.copy_(torch.where(T >= 0, to[T.clamp(min=0).long()], -1))
    half = s["pairs"].shape[0]
    s["pairs"].copy_(torch.stack([src[:half], dst[:half]], 1))
    s["n_pairs"].copy_(n.view(1))
    s["bits"].copy_(_free_bits(ref))


def _plain_copy(s):
    """Pages of all layers; entries past n_pairs repeat the first pair, or copy page 0 onto itself."""
    p = s["pairs"][:s["most"]].long()
    first = torch.where(s["n_pairs"] > 0, p[0], 0)
    live = torch.arange(p.shape[0], device="cuda") < s["n_pairs"]
    p = torch.where(live[:, None], p, first)
    s["pool"][:, p[:, 1]] = s["pool"][:, p[:, 0]]


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    if case["op"] not in ("append", "attention"):
        return None
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)


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


def _round4(x, one):
    """The nearest of the 4-bit values to x / one, ties to the even code (distances in units of `one`: exact)."""
    v = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    far = (x.abs()[..., None] - v * one[..., None]).abs()
    best = far.amin(-1, keepdim=True)
    pick = torch.where(far == best, torch.arange(8, device="cuda"), 99)
    even = torch.where(pick % 2 == 0, pick, 99).amin(-1)
    return v[torch.where(even < 99, even, pick.amin(-1))] * torch.sign(x)


def _exact_append(s):
    c = s["case"]
    Hkv, P, D = c["Hkv"], c["page"], c["D"]
    lens, ells = _lens(c), _ells(c)
    q = s["q_out"].double()
    if c["fmt"] == BF16:
        pool = s["pool"].view(torch.bfloat16).double()
        page = pool.view(-1, Hkv, 2, P // 16, 16 * D)
        e = torch.arange(D, device="cuda")
    else:
        kr, vr = s["k_read"].double(), s["v_read"].double()
    row = 0
    for r in range(c["R"]):
        for i in range(ells[r] + 1):
            p = lens[r] + i
            q[row] = _turn(s["q"][row], s["wq"], p, s)
            k, v = _turn(s["k"][row], s["wk"], p, s), s["v"][row].double()
            if c["fmt"] == BF16:
                at = page[int(s["table"][r, p // P])]
                t, b = p % 16, p % P // 16
                at[:, 0, b, (e // 8 * 16 + t) * 8 + e % 8] = k
                at[:, 1, b, (t // 8 * D + e) * 8 + t % 8] = v
            else:
                g = k.view(Hkv, D // 32, 32)
                top = g.abs().amax(-1, keepdim=True)
                step = torch.exp2(torch.frexp(top)[1].double() - 3)   # top / step in [4, 8)
                step = torch.where(top > 7 * step, 2 * step, step)
                kr[r, i] = (_round4(g, step) * step).view(Hkv, D)
                top = v.abs().amax(-1, keepdim=True)
                vr[r, i] = _round4(6 * v, top) * top / 6
            row += 1
    return {"q": q, "pool": pool} if c["fmt"] == BF16 else {"q": q, "k": kr, "v": vr}


def _exact_attention(s):
    c = s["case"]
    Hq, Hkv, D, P = c["Hq"], c["Hkv"], c["D"], c["page"]
    lens, ells = _lens(c), _ells(c)
    if sum(n * (e + 1) for n, e in zip(lens, ells)) * Hq * D > 3e11:
        return None
    out, lse = s["out"].double(), s["lse"].double()
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    row = 0
    for r in range(c["R"]):
        n = ells[r] + 1
        if n == 0:
            continue
        N = lens[r] + n
        page = s["pool"][s["table"][r, :_up(N, P)].long()]
        if c["fmt"] == BF16:
            x = page.view(torch.bfloat16).view(-1, Hkv, 2, P // 16, 16 * D)
            k = x[:, :, 0].reshape(-1, Hkv, P // 16, D // 8, 16, 8).permute(1, 0, 2, 4, 3, 5).reshape(Hkv, -1, D)
            v = x[:, :, 1].reshape(-1, Hkv, P // 16, 2, D, 8).permute(1, 0, 2, 3, 5, 4).reshape(Hkv, -1, D)
            k, v = k[:, :N].double(), v[:, :N].double()
        else:
            x = page.view(page.shape[0], Hkv, -1)
            a, b = P * D // 2, P * D // 32
            k = x[:, :, :a].reshape(-1, Hkv, P // 16, D // 32, 16, 16).permute(1, 0, 2, 4, 3, 5).reshape(Hkv, -1, D // 2)
            k = torch.stack([lut[(k & 15).int()], lut[(k >> 4).int()]], -1).view(Hkv, -1, D // 32, 32)
            sc = x[:, :, a:a + b].reshape(-1, Hkv, P, D // 32).transpose(0, 1).reshape(Hkv, -1, D // 32, 1)
            k = (k * torch.exp2(sc.double() - 127)).view(Hkv, -1, D)[:, :N]
            v = x[:, :, a + b:2 * a + b].reshape(-1, Hkv, P // 16, 2, 32, D // 32, 4)
            v = torch.stack([lut[(v & 15).int()], lut[(v >> 4).int()]], -1).flatten(-2)
            v = v.permute(1, 0, 2, 3, 6, 5, 4).reshape(Hkv, -1, D)
            sc = x[:, :, 2 * a + b:].contiguous().view(torch.float32).transpose(0, 1).reshape(Hkv, -1, 1)
            v = (v * sc.double())[:, :N]
        q = s["q"][row:row + n].double().view(n, Hkv, Hq // Hkv, D).permute(1, 0, 2, 3).reshape(Hkv, -1, D)
        score = torch.bmm(q, k.transpose(1, 2).contiguous()).view(Hkv, n, Hq // Hkv, N) / math.sqrt(D)
        for i in range(n):
            p = lens[r] + i
            score[:, i, :, p + 1:] = -math.inf
            if c["window"]:
                score[:, i, :, min(c["sinks"], p):max(0, p - c["window"] + 1)] = -math.inf
        z = torch.logsumexp(score, -1)
        o = torch.bmm(torch.exp(score - z[..., None]).view(Hkv, -1, N), v.contiguous())
        out[row:row + n] = o.view(Hkv, n, Hq // Hkv, D).permute(1, 0, 2, 3).reshape(n, Hq, D)
        lse[row:row + n] = z.permute(1, 0, 2).reshape(n, Hq)
        row += n
    return {"out": out, "lse": lse}
