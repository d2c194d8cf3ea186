"""dspark_cache_attention against the float64 oracle, with the error bounds
that cache_cases.attention_tolerance derives.  Bytes of the pools that no
token was written to are all ones (NaNs), so a read of them shows."""

import sys

import numpy as np
import pytest

from cache_cases import BF16, FP4, attention_tolerance, bf, build
from oracle import cache as OC
from semi_ar_draft_round_amd.workloads import bf16_to_f32

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from semi_ar_draft_round_amd import binding
    binding.load_library()
    return torch.device("cuda:0")


def t16(bits, dev):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).to(dev)


def back(t):
    return bf16_to_f32(t.cpu().view(torch.int16).numpy().view(np.uint16)).astype(np.float64)


class Case:
    def __init__(self, dev, fmt, lens, ells, Hq, Hkv, D, P, gamma, window=0, sinks=0, packed=True, seed=1, peak=1.0,
                 max_pages=None, scale=None):
        rng = np.random.default_rng(seed)
        self.__dict__.update(fmt=fmt, lens=lens, ells=ells, Hq=Hq, Hkv=Hkv, D=D, P=P, gamma=gamma, window=window,
                             sinks=sinks, scale=D ** -0.5 if scale is None else scale, dev=dev)
        n = [min(max(e, -1), gamma) + 1 for e in ells]
        total = [a + b for a, b in zip(lens, n)]
        mp = max(1, max(-(-t // P) for t in total)) if max_pages is None else max_pages
        self.npool, self.ntable, self.ks, self.vs = build(rng, fmt, total, Hkv, D, P, mp)
        first = (np.cumsum([0] + n)[:-1] + 1).tolist() if packed else [r * (gamma + 1) for r in range(len(lens))]
        self.rows = sum(n) + 2 if packed else len(lens) * (gamma + 1)
        self.first, self.n = first, n
        qb, self.nq = bf(rng.standard_normal((self.rows, Hq, D)) * peak)
        self.q = t16(qb, dev)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
        self.row0 = i32(first) if packed else None
        self.ell, self.length = i32(ells), i32(lens)
        self.pool, self.table = torch.from_numpy(self.npool).to(dev), torch.from_numpy(self.ntable).to(dev)

    def call(self, out=None, lse=None, **kw):
        from semi_ar_draft_round_amd import binding as B
        return B.dspark_cache_attention(self.q, self.pool, self.table, self.length, self.ell, self.gamma, fmt=self.fmt,
                                        page=self.P, heads_kv=self.Hkv, scale=self.scale, window=self.window,
                                        sinks=self.sinks, row0=self.row0, out=out, lse=lse, **kw)

    def check(self, have=None, vs=None):
        out = torch.full((self.rows, self.Hq, self.D), 5.0, dtype=torch.bfloat16, device=self.dev)
        lse = torch.full((self.rows, self.Hq), 5.0, dtype=torch.float32, device=self.dev)
        self.call(out, lse)
        torch.cuda.synchronize()
        o, z = back(out), lse.cpu().numpy().astype(np.float64)
        mine = np.zeros(self.rows, dtype=bool)
        worst = 0.0
        for r, (f, n) in enumerate(zip(self.first, self.n)):
            if n == 0:
                continue
            mine[f:f + n] = True
            pos = self.lens[r] + np.arange(n)
            h = None if have is None else have[r]
            v = self.vs[r] if vs is None else vs[r]
            want, wz = OC.attention(self.nq[f:f + n], self.ks[r], v, pos, self.scale, self.window, self.sinks, h)
            to, tz = attention_tolerance(self.nq[f:f + n], self.ks[r], v, pos, self.scale, self.window, self.sinks, want,
                                         h)
            bad = ~np.isfinite(want)
            assert np.array_equal(np.isnan(want), np.isnan(o[f:f + n]))
            err = np.abs(np.where(bad, 0, o[f:f + n]) - np.where(bad, 0, want))
            assert np.all(err <= to), (r, float((err / to).max()))
            worst = max(worst, float((err / to).max()))
            gone = np.isneginf(wz)
            assert np.array_equal(gone, np.isneginf(z[f:f + n]))
            assert np.all(np.abs(np.where(gone, 0, z[f:f + n]) - np.where(gone, 0, wz)) <= tz + 2.0 ** -22 * np.abs(
                np.where(gone, 0, wz)))
        assert np.all(o[~mine] == 5.0) and np.all(z[~mine] == 5.0)       # rows of nobody
        say(f"  worst error {worst:.3f} of its bound")


SHAPES = [  # lens, ells, Hq, Hkv, D, P, gamma, window, sinks, packed
    ([0], [0], 1, 1, 64, 16, 0, 0, 0, False),                       # the first token alone
    ([1], [0], 4, 2, 128, 64, 0, 0, 0, False),
    ([0, 5, 31, 32, 33], [16, 0, 16, 7, -1], 8, 2, 128, 16, 16, 0, 0, True),
    ([700, 64, 129, 0], [16, 3, 1, 0], 14, 2, 128, 64, 16, 0, 0, True),   # groups of seven
    ([255, 256, 257], [4, 4, 4], 6, 6, 64, 32, 4, 0, 0, False),     # no groups
    ([300, 90], [64, 64], 5, 1, 256, 128, 64, 0, 0, True),          # five heads on one
    ([1500], [0], 8, 8, 64, 16, 0, 0, 0, False),                    # long and split
    ([400, 40, 3], [16, 16, 16], 8, 2, 128, 16, 16, 100, 4, True),  # window and first tokens
    ([400, 140, 30], [16, 9, 16], 4, 4, 64, 32, 16, 1, 0, True),    # only itself
    ([513, 200], [16, 16], 16, 2, 128, 64, 16, 64, 70, True),       # first tokens past a tile
    ([500, 20], [5, 5], 4, 2, 256, 16, 5, 33, 1000, True),          # first tokens cover everything
    ([900], [300], 2, 1, 64, 64, 300, 130, 3, True),                # a prompt's chunk under a window
    ([0, 77], [200, 150], 3, 3, 128, 16, 200, 0, 0, True),          # chunks over an empty cache
    ([60, 61], [1, 0], 40, 1, 128, 16, 1, 0, 0, True),              # forty heads on one
]


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(x) for x in s))
def test_attention_against_oracle(shape, fmt, dev):
    say(f"[attention] fmt {fmt} {shape}")
    lens, ells, Hq, Hkv, D, P, gamma, window, sinks, packed = shape
    Case(dev, fmt, lens, ells, Hq, Hkv, D, P, gamma, window, sinks, packed).check()


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_peaked_scores(fmt, D, dev):
    """Scores in the hundreds: the running maximum moves at every tile."""
    say(f"[attention] peaked {fmt} {D}")
    Case(dev, fmt, [333, 40], [16, 2], 8, 2, D, 32, 16, peak=60.0, seed=4).check()
    Case(dev, fmt, [333], [3], 8, 2, D, 32, 3, scale=0.0, seed=5).check()      # every visible token alike
    Case(dev, fmt, [333], [3], 8, 2, D, 32, 3, scale=-0.2, seed=6).check()


@pytest.mark.parametrize("fmt", [BF16, FP4])
def test_missing_pages(fmt, dev):
    """Pages without a table entry, or with one out of range, are invisible;
    a row that sees nothing is zero with lse -inf."""
    say(f"[attention] missing pages {fmt}")
    for window, sinks in ((0, 0), (50, 20)):
        c = Case(dev, fmt, [200, 90, 40, 10], [16, 3, 0, 5], 8, 2, 128, 16, 16, window, sinks)
        t = c.ntable.copy()
        t[0, 2:5] = -1
        t[0, 12] = 10 ** 6
        t[1, :] = -1                      # nothing left at all
        t[2, -1] = -7
        t[3, 0] = -1                      # its only page
        have = []
        for r in range(4):
            ok = (t[r] >= 0) & (t[r] < c.npool.shape[0])
            have.append(np.repeat(ok, c.P)[:c.ks[r].shape[0]])
        c.table = torch.from_numpy(t).to(dev)
        c.check(have=have)


def test_what_is_invisible_has_no_effect(dev):
    """Infinities, NaNs and the type's lowest value in tokens that a row does
    not see (later rows of the block, tokens before the window, tokens behind
    the last row in its page) change nothing, bit for bit."""
    say("[attention] invisible")
    from semi_ar_draft_round_amd import binding as B
    for D, P, Hq, Hkv, window, sinks in ((128, 64, 8, 2, 0, 0), (64, 16, 4, 4, 40, 3), (256, 32, 7, 1, 21, 0)):
        lens, gamma = [130, 77, 3], 16
        c = Case(dev, BF16, lens, [16, 9, 16], Hq, Hkv, D, P, gamma, window, sinks, seed=9)
        out = torch.zeros((c.rows, Hq, D), dtype=torch.bfloat16, device=dev)
        lse = torch.zeros((c.rows, Hq), dtype=torch.float32, device=dev)
        c.call(out, lse)
        # rewrite row m and everything after it, and all before the window, of every request
        m = 5
        poison = [float("inf"), float("-inf"), float("nan"), -3.3895313892515355e38]
        pool = c.pool.clone()
        for r in range(3):
            first, last = lens[r] + m, lens[r] + c.n[r]
            hidden = list(range(first, last))
            if window:
                hidden += [t for t in range(0, max(0, lens[r] - window + 1)) if t >= sinks]
            pages = pool.view(torch.bfloat16).view(pool.shape[0], Hkv, 2, P // 16, 16 * D)
            for x, t in enumerate(hidden):
                p, u = int(c.table[r, t // P]), t % P
                e = torch.arange(D, device=dev)
                pages[p, :, 0, u // 16, (e // 8 * 16 + u % 16) * 8 + e % 8] = poison[x % 4]
                pages[p, :, 1, u // 16, ((u % 16) // 8 * D + e) * 8 + u % 8] = poison[(x + 1) % 4]
        keep = c.pool
        c.pool = pool
        out2, lse2 = torch.zeros_like(out), torch.zeros_like(lse)
        c.call(out2, lse2)
        torch.cuda.synchronize()
        rows = [f + i for f, n in zip(c.first, c.n) for i in range(min(m, n))]
        assert torch.equal(out[rows], out2[rows]) and torch.equal(lse[rows], lse2[rows])
        c.pool = keep
    # the same for 4-bit pages: NaN scales in hidden tokens
    c = Case(dev, FP4, [130, 77], [16, 9], 8, 2, 128, 64, 16, 40, 3, seed=9)
    out, lse = torch.zeros((c.rows, 8, 128), dtype=torch.bfloat16, device=dev), torch.zeros((c.rows, 8), device=dev)
    c.call(out, lse)
    hb = c.pool.shape[1] // 2
    view = c.pool.view(c.pool.shape[0], 2, hb)
    for r, n in enumerate(c.lens):
        for t in list(range(n + 5, n + c.n[r])) + list(range(3, n - 39)):
            p, u = int(c.table[r, t // 64]), t % 64
            view[p, :, 64 * 64 + u * 4:64 * 64 + u * 4 + 4] = 255
            view[p, :, 64 * 132 + u * 4:64 * 132 + u * 4 + 4] = 255
    out2, lse2 = torch.zeros_like(out), torch.zeros_like(lse)
    c.call(out2, lse2)
    rows = [f + i for f, n in zip(c.first, c.n) for i in range(5)]
    assert torch.equal(out[rows], out2[rows]) and torch.equal(lse[rows], lse2[rows])


def test_visible_infinities(dev):
    """A visible infinite value reaches the rows that see it and no other; a
    visible NaN score makes its rows NaN."""
    say("[attention] visible infinities")
    c = Case(dev, BF16, [100], [16], 4, 2, 128, 32, 16, seed=10)
    p, u = int(c.table[0, 104 // 32]), 104 % 32
    pages = c.pool.view(torch.bfloat16).view(c.pool.shape[0], 2, 2, 2, 16 * 128)
    pages[p, 0, 1, u // 16, ((u % 16) // 8 * 128 + 17) * 8 + u % 8] = float("inf")
    out, _ = c.call()
    o = back(out)[c.first[0]:c.first[0] + 17]
    assert np.isfinite(o[:4]).all()
    assert np.isposinf(o[4:, :2, 17]).all()
    o[4:, :2, 17] = 0
    assert np.isfinite(o).all()
    e = torch.arange(128, device=dev)
    pages[p, 1, 0, u // 16, (e // 8 * 16 + u % 16) * 8 + e % 8] = float("nan")
    out, _ = c.call()
    o = back(out)[c.first[0]:c.first[0] + 17]
    assert np.isfinite(o[:4]).all() and np.isnan(o[4:, 2:]).all() and np.isfinite(o[4:, :2, :17]).all()


@pytest.mark.parametrize("fmt", [BF16, FP4])
def test_offsets_past_32_bits(fmt, dev):
    """A pool of more than 4 GB whose pages in use lie at its end."""
    from semi_ar_draft_round_amd import binding as B
    say(f"[attention] far pages {fmt}")
    c = Case(dev, fmt, [200, 70], [3, 16], 8, 2, 128, 128, 16, seed=12)
    nb = c.npool.shape[1]
    n = (5 << 30) // nb
    big = torch.empty((n, nb), dtype=torch.uint8, device=dev)
    m = c.npool.shape[0]
    big[n - m:] = c.pool
    small = c.pool
    c.pool = big
    c.table = torch.where(c.table >= 0, c.table + (n - m), c.table).to(torch.int32)
    c.check()
    del small


def test_long_cache_is_split_and_joined(dev):
    """One request over 40,000 tokens against float64 on the device."""
    from semi_ar_draft_round_amd import binding as B
    say("[attention] long")
    Hq, Hkv, D, P, N, n = 8, 2, 128, 64, 40_000, 17
    g = torch.Generator(device=dev).manual_seed(3)
    pages = -(-N // P)
    pool = torch.randn(pages * Hkv * 2 * P * D, generator=g, device=dev).to(torch.bfloat16)
    table = torch.randperm(pages, generator=g, device=dev).to(torch.int32)[None].contiguous()
    q = torch.randn(n, Hq, D, generator=g, device=dev).to(torch.bfloat16)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    lse = torch.zeros(n, Hq, device=dev)
    out, _ = B.dspark_cache_attention(q, pool.view(torch.uint8).view(pages, -1), table, i32([N - n]), i32([n - 1]), n - 1,
                                      fmt=BF16, page=P, heads_kv=Hkv, lse=lse)
    x = pool.view(pages, Hkv, 2, P // 16, 16 * D)[table[0].long()]
    k = x[:, :, 0].reshape(-1, Hkv, P // 16, D // 8, 16, 8).permute(1, 0, 2, 4, 3, 5).reshape(Hkv, -1, D).double()
    v = x[:, :, 1].reshape(-1, Hkv, P // 16, 2, D, 8).permute(1, 0, 2, 3, 5, 4).reshape(Hkv, -1, D).double()
    s = torch.bmm(q.double().view(n, Hkv, -1, D).permute(1, 0, 2, 3).reshape(Hkv, -1, D), k.transpose(1, 2).contiguous())
    s = s.view(Hkv, n, -1, pages * P) * D ** -0.5
    for i in range(n):
        s[:, i, :, N - n + i + 1:] = float("-inf")
    z = torch.logsumexp(s, -1)
    p = torch.exp(s - z[..., None]).view(Hkv, -1, pages * P)
    want = torch.bmm(p, v.contiguous()).view(Hkv, n, -1, D).permute(1, 0, 2, 3).reshape(n, Hq, D)
    mean_abs = torch.bmm(p, v.abs().contiguous()).view(Hkv, n, -1, D).permute(1, 0, 2, 3).reshape(n, Hq, D)
    # as attention_tolerance; |q| |k| of a score is below 200 here, times D^-1/2
    delta = 2 * (D + 8) * 2.0 ** -24 * 200 * D ** -0.5
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + delta + (N + 64) * 2.0 ** -24) * mean_abs
    assert bool(((out.double() - want).abs() <= tol).all())
    assert float((lse.double() - z.permute(1, 0, 2).reshape(n, Hq)).abs().max()) <= delta + (N + 64) * 2.0 ** -24


@pytest.mark.parametrize("fmt", [BF16, FP4])
def test_streams_graphs_and_repeats(fmt, dev):
    """Twice, on a side stream, two calls at once with workspaces of their
    own, a dirty workspace, and captured with eager calls between the
    replays: the same bits."""
    from semi_ar_draft_round_amd import binding as B
    say(f"[attention] streams {fmt}")
    a = Case(dev, fmt, [2000, 333, 40], [16, 16, 3], 8, 2, 128, 64, 16, seed=20)
    b = Case(dev, fmt, [1500, 700], [2, 16], 14, 2, 128, 32, 16, 200, 4, seed=21)
    want = [x.call(lse=torch.zeros((x.rows, x.Hq), device=dev)) for x in (a, b)]
    live = [[f + i for f, n in zip(x.first, x.n) for i in range(n)] for x in (a, b)]

    def same(x, got):
        i = 0 if x is a else 1
        assert torch.equal(want[i][0][live[i]], got[0][live[i]]) and torch.equal(want[i][1][live[i]], got[1][live[i]])

    for x in (a, b):
        size = B.dspark_cache_workspace_size(B.CACHE_WS_ATTENTION, len(x.lens), x.gamma, x.Hq, x.Hkv, x.D)
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=dev)
        same(x, x.call(lse=torch.zeros((x.rows, x.Hq), device=dev), ws=ws))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        torch.cuda.synchronize()
        for x, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                got.append(x.call(lse=torch.zeros((x.rows, x.Hq), device=dev)))
        torch.cuda.synchronize()
        same(a, got[0])
        same(b, got[1])
    g = torch.cuda.CUDAGraph()
    outs = [(torch.zeros_like(want[i][0]), torch.zeros_like(want[i][1])) for i in range(2)]
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        a.call(*outs[0])
        b.call(*outs[1])
    for _ in range(4):
        for o in outs:
            o[0].zero_(), o[1].zero_()
        g.replay()
        same(a, a.call(lse=torch.zeros((a.rows, a.Hq), device=dev)))
        torch.cuda.synchronize()
        same(a, outs[0])
        same(b, outs[1])


LARGE = [  # lens, ells, Hq, Hkv, D, P, gamma: how the work is dealt
    ([40_000, 9_001, 33, 25_000, 17_000], [16, 3, 0, 16, 9], 16, 8, 64, 64, 16),  # equal runs whatever the requests
    ([16_383] * 8, [0] * 8, 16, 8, 128, 64, 0),               # whole parts of heads, an even number
    ([12_000, 11_990, 12_011], [5, 5, 5], 8, 8, 128, 16, 5),  # an odd number
    ([6_000] * 8, [16] * 8, 32, 8, 64, 128, 16),              # four row tiles a head
    ([3_000, 10, 2_500], [-1, 16, -1], 4, 2, 128, 32, 16),    # few heads, most requests idle
    ([2_000] * 6, [16] * 6, 8, 2, 256, 64, 16),
    (list(range(40)) * 103, [0, -1, 0] * 1373, 2, 1, 64, 16, 0),                  # 4096 requests at most: 4119 cut below
]


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("case", LARGE, ids=["runs", "parts", "odd-parts", "row-tiles", "idle", "d256", "r4096"])
def test_work_shared_out(case, fmt, dev):
    """Batches large enough for every way of dealing the work out, against
    float64 on the device over the values that dspark_cache_read gives (of
    4 bits V rounded to bf16, which adds 2^-8 of sum_j p_j |v_j|)."""
    from semi_ar_draft_round_amd import binding as B
    lens, ells, Hq, Hkv, D, P, gamma = case
    lens, ells = lens[:4096], ells[:4096]
    say(f"[attention] {len(lens)} requests, fmt {fmt}, D {D}")
    R, T = len(lens), max(lens) + gamma + 1
    g = torch.Generator(device=dev).manual_seed(17)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    mp = -(-T // P)
    pool = torch.full((R * mp, B.dspark_cache_page_bytes(fmt, Hkv, D, P)), 0xFF, dtype=torch.uint8, device=dev)
    table = torch.randperm(R * mp, generator=g, device=dev).to(torch.int32).view(R, mp)
    total = [n + max(e, -1) + 1 for n, e in zip(lens, ells)]
    C = min(1024, T)
    for at in range(0, T, C):
        x = torch.randn((R * C, 1 + 2 * Hkv, D), generator=g, device=dev).to(torch.bfloat16)
        B.dspark_cache_append(x[:, :1], x[:, 1:1 + Hkv], x[:, 1 + Hkv:], pool, table, i32([min(at, t) for t in total]),
                              i32([min(t - at, C) - 1 if t > at else -1 for t in total]), C - 1, fmt=fmt, page=P)
    n = [e + 1 for e in ells]
    first = np.cumsum([0] + n)[:-1].tolist()
    q = torch.randn((sum(n), Hq, D), generator=g, device=dev).to(torch.bfloat16)
    lse = torch.zeros((sum(n), Hq), device=dev)
    out, _ = B.dspark_cache_attention(q, pool, table, i32(lens), i32(ells), gamma, fmt=fmt, page=P, heads_kv=Hkv,
                                      row0=i32(first), lse=lse)
    again, _ = B.dspark_cache_attention(q, pool, table, i32(lens), i32(ells), gamma, fmt=fmt, page=P, heads_kv=Hkv,
                                        row0=i32(first))
    assert torch.equal(out, again)
    scale, worst = D ** -0.5, 0.0
    for r in range(R):
        if n[r] == 0 or (R > 100 and r % 7):
            continue
        N = total[r]
        k, v = B.dspark_cache_read(pool, table[r:r + 1].contiguous(), None, i32([N]), N, fmt=fmt, page=P, heads_kv=Hkv,
                                   dim=D)
        k, v = (y[0].double().permute(1, 0, 2).contiguous() for y in (k, v))
        mine = slice(first[r], first[r] + n[r])
        x = q[mine].double().view(n[r], Hkv, -1, D).permute(1, 0, 2, 3).reshape(Hkv, -1, D)
        s = (torch.bmm(x, k.transpose(1, 2).contiguous()) * scale).view(Hkv, n[r], -1, N)
        for i in range(n[r]):
            s[:, i, :, lens[r] + i + 1:] = float("-inf")
        z = torch.logsumexp(s, -1)
        p = torch.exp(s - z[..., None]).view(Hkv, -1, N)
        rows = lambda y: y.view(Hkv, n[r], -1, D).permute(1, 0, 2, 3).reshape(n[r], Hq, D)
        want, mean_abs = rows(torch.bmm(p, v)), rows(torch.bmm(p, v.abs().contiguous()))
        # as attention_tolerance, sum |q k| at most the product of the norms
        delta = 2 * (D + 8) * 2.0 ** -24 * float(x.norm(dim=-1).max() * k.norm(dim=-1).max()) * scale
        rest = delta + (N + 64) * 2.0 ** -24
        half = 2.0 ** -8
        tol = half * want.abs() + (half * (1 + half) + rest + (half if fmt == FP4 else 0)) * mean_abs + 1e-30
        err = (out[mine].double() - want).abs()
        assert bool((err <= tol).all()), (r, float((err / tol).max()))
        worst = max(worst, float((err / tol).max()))
        zr = z.permute(1, 0, 2).reshape(n[r], Hq)
        assert bool(((lse[mine].double() - zr).abs() <= rest + 1e-6 + 2.0 ** -22 * zr.abs()).all())
    say(f"  worst error {worst:.3f} of its bound")
