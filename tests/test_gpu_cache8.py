"""8-bit pages: append, read and attention against the float64 oracle.  Codes
and scales are compared exactly (keys are fp64 on both sides, and a key within
2^-50 of a border between two codes does not come up), attention within the
bounds that cache_cases.attention_tolerance derives."""

import sys

import numpy as np
import pytest

from cache8_cases import FP8, build8, dense, page_bytes8
from cache_cases import bf
from oracle import cache as OC
from semi_ar_draft_round_amd.workloads import bf16_to_f32
from test_gpu_cache_attention import SHAPES, Case, back, t16

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


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


class Cache8:
    """A pool of 8-bit pages beside what the oracle says it holds."""

    def __init__(self, dev, R, Hq, Hkv, D, P, max_pages, norm=True, rot=None, adjacent=False, seed=1):
        rng = np.random.default_rng(seed)
        self.__dict__.update(dev=dev, R=R, Hq=Hq, Hkv=Hkv, D=D, P=P, rng=rng, adjacent=adjacent)
        self.N = R * max_pages + 2
        self.ntable = rng.permutation(self.N)[:R * max_pages].reshape(R, max_pages).astype(np.int32)
        self.npool = np.full((self.N, page_bytes8(Hkv, D, P)), 0xFF, np.uint8)
        self.table, self.pool = torch.from_numpy(self.ntable).to(dev), torch.from_numpy(self.npool).to(dev)
        self.want = self.npool.copy()       # what rolled-back tokens left stays until it is written over
        self.K = [[OC.Rows8(D) for _ in range(Hkv)] for _ in range(R)]
        self.V = [[OC.Rows8(D) for _ in range(Hkv)] for _ in range(R)]
        rot = D if rot is None else rot
        self.freq = 1e4 ** (-2.0 * np.arange(rot // 2) / max(rot, 1))
        self.nw = [bf(1 + 0.3 * rng.standard_normal(D))[1] if norm else None for _ in range(2)]
        self.w = [None if w is None else t16(bf(w)[0], dev) for w in self.nw]

    def rows(self, n, H, spread):
        b, x = bf(self.rng.standard_normal((n, H, self.D)) * spread)
        return b, x

    def append(self, lens, ells, gamma, kspread=1.0, vspread=1.0, packed=True, edit=None, table=None):
        """One call; the oracle's rows of requests whose page exists follow."""
        from semi_ar_draft_round_amd import binding as B
        n = [min(max(e, -1), gamma) + 1 for e in ells]
        first = (np.cumsum([0] + n)[:-1] + 1).tolist() if packed else [r * (gamma + 1) for r in range(self.R)]
        rows = sum(n) + 2 if packed else self.R * (gamma + 1)
        (qb, q), (kb, k), (vb, v) = (self.rows(rows, h, s) for h, s in ((self.Hq, 1), (self.Hkv, kspread),
                                                                        (self.Hkv, vspread)))
        if edit:
            edit(kb, k, vb, v, first)
        out = torch.full((rows, self.Hq, self.D), 5.0, dtype=torch.bfloat16, device=self.dev)
        # keys and values as views of one wider row
        both = torch.cat([t16(kb, self.dev), t16(vb, self.dev)], dim=1)
        B.dspark_cache_append(t16(qb, self.dev), both[:, :self.Hkv], both[:, self.Hkv:], self.pool,
                              self.table if table is None else table, i32(lens, self.dev), i32(ells, self.dev), gamma,
                              fmt=FP8, page=self.P, wq=self.w[0], wk=self.w[1],
                              freq=torch.from_numpy(self.freq).to(self.dev) if len(self.freq) else None,
                              adjacent=self.adjacent, row0=i32(first, self.dev) if packed else None, q_out=out)
        torch.cuda.synchronize()
        got, mine = back(out), np.zeros(rows, bool)
        for r in range(self.R):
            f, m = first[r], n[r]
            if m == 0 or lens[r] < 0:
                continue
            mine[f:f + m] = True
            pos = lens[r] + np.arange(m)
            turn = lambda x, w: OC.rotate(OC.norm(x, w, 1e-6), pos, self.freq, self.adjacent)
            # fp32 norm and rotation: D + 16 roundings of 2^-24 on the magnitudes, then bf16 (2^-8)
            want = turn(q[f:f + m], self.nw[0])
            mag = np.abs(want).max(-1, keepdims=True) * 2
            assert np.all(np.abs(got[f:f + m] - want) <= np.abs(want) * 2.0 ** -8 + mag * (self.D + 16) * 2.0 ** -24)
            kk = turn(k[f:f + m], self.nw[1])
            for h in range(self.Hkv):
                self.K[r][h].append(lens[r], kk[:, h])
                self.V[r][h].append(lens[r], v[f:f + m, h])
            if table is None:
                OC.write_pages8(self.K[r], self.V[r], self.ntable[r], self.P, self.want)
        assert np.all(got[~mine] == 5.0)

    def check(self):
        """Codes and scales byte by byte, nothing else in the pool written."""
        want, got = self.want, self.pool.cpu().numpy()
        # a NaN code may have either sign, a zero too
        hb = page_bytes8(1, self.D, self.P)
        codes = lambda x: x.reshape(self.N, self.Hkv, hb)[:, :, :2 * self.P * self.D]
        g, w = codes(got), codes(want)
        same = (g == w) | ((g & 127) == 127) & ((w & 127) == 127) | ((g & 127) == 0) & ((w & 127) == 0)
        assert same.all(), np.argwhere(~same)[:5]
        assert np.array_equal(got.reshape(self.N, self.Hkv, hb)[:, :, 2 * self.P * self.D:],
                              want.reshape(self.N, self.Hkv, hb)[:, :, 2 * self.P * self.D:])

    def check_read(self, lens):
        from semi_ar_draft_round_amd import binding as B
        T = max(max(lens), 1)
        k, v = B.dspark_cache_read(self.pool, self.table, None, i32(lens, self.dev), T, fmt=FP8, page=self.P,
                                   heads_kv=self.Hkv, dim=self.D)
        k, v = back(k), back(v)
        for r, n in enumerate(lens):
            if n:
                assert np.array_equal(k[r, :n], dense(self.K[r])[:n], equal_nan=True)
                assert np.array_equal(v[r, :n], dense(self.V[r])[:n], equal_nan=True)
            assert np.all(k[r, n:] == 0) and np.all(v[r, n:] == 0)


@pytest.mark.parametrize("D,P,rot,adjacent,norm", [(64, 16, 64, False, True), (128, 64, 128, False, True),
                                                   (128, 32, 64, True, False), (256, 128, 256, False, True),
                                                   (256, 16, 96, False, True), (64, 128, 0, False, False),
                                                   (128, 16, 128, True, True)])
def test_append_and_read(D, P, rot, adjacent, norm, dev):
    """Rounds with rows rolled back, blocks that grow and that do not."""
    say(f"[cache8] append {D} {P} {rot} {adjacent} {norm}")
    c = Cache8(dev, 4, 6, 3, D, P, 256 // P, norm, rot, adjacent, seed=D + P)
    lens = [0, 0, 0, 0]
    for gamma, ells, kept, spread in ((40, [0, 40, 16, -1], [0, 33, 14, 0], 1.0), (16, [16, 2, 0, 16], [16, 1, 0, 15], 3.0),
                                      (16, [16, 16, 16, 16], [0, 16, 5, 2], 0.01), (4, [-1, 4, 3, 0], [0, 4, 0, 0], 100.0),
                                      (70, [70, 15, 64, 70], [70, 15, 64, 31], 1.0)):
        c.append(lens, ells, gamma, kspread=spread, vspread=spread, packed=gamma != 4)
        after = [n + e + 1 for n, e in zip(lens, ells)]
        c.check()
        c.check_read(after)
        lens = [n + (k + 1 if e >= 0 else 0) for n, e, k in zip(lens, ells, kept)]


def test_one_token_at_a_time(dev):
    say("[cache8] tokens")
    c = Cache8(dev, 2, 2, 5, 128, 16, 3, seed=5)
    for n in range(35):
        c.append([n, n // 2 * 2], [0, 0 if n % 2 else -1], 0, kspread=1 + n % 5, vspread=2.0 ** (n % 11))
        if n % 2:
            c.append([n + 1, n - 1], [-1, 1], 1)     # two rows over the one that is there
            c.check()
    c.check_read([35, 34])


def test_every_value_between_the_codes(dev):
    """All bf16 numbers up to 448 as values, under a scale of 1: every tie and
    both its neighbours, subnormal codes, what rounds to zero."""
    say("[cache8] roundings")
    D = 64
    bits = np.arange(0x3880, 0x43E1).astype(np.uint16)                 # 2^-14 .. 448
    x = np.concatenate([bits, bits | 0x8000])
    T = -(-len(x) // (D - 1))
    rows = np.zeros((T, 1, D), np.uint16)
    rows[:, 0, 0] = 0x43E0                                             # 448 in every row
    flat = np.zeros(T * (D - 1), np.uint16)
    flat[:len(x)] = x
    rows[:, 0, 1:] = flat.reshape(T, D - 1)

    def edit(kb, k, vb, v, first):
        vb[first[0]:first[0] + T] = rows
        v[first[0]:first[0] + T] = bf16_to_f32(rows)

    c = Cache8(dev, 1, 1, 1, D, 128, -(-T // 128), norm=False, rot=0, seed=6)
    c.append([0], [T - 1], T - 1, edit=edit)
    assert all(e == 0 for e in c.V[0][0].e)
    c.check()
    c.check_read([T])


@pytest.mark.parametrize("value", [0.0, 2.0 ** -133, 2.0 ** -120, 3.3895313892515355e38, 1.7e38, 2.9e38])
def test_far_magnitudes(value, dev):
    """Zeros, the least and the largest numbers of bf16 as keys and values;
    then ordinary rows join the block."""
    say(f"[cache8] magnitude {value}")

    def edit(kb, k, vb, v, first):
        b, x = bf(np.full((3, 1, 128), value) * np.where(np.arange(128) % 3, 1, -1))
        for bits, y in ((kb, k), (vb, v)):
            bits[first[0]:first[0] + 3], y[first[0]:first[0] + 3] = b, x

    for norm, rot in ((False, 0), (False, 128)):
        c = Cache8(dev, 1, 1, 1, 128, 16, 2, norm=norm, rot=rot, seed=7)
        c.append([0], [2], 2, edit=edit)
        c.check()
        c.append([3], [8], 8)
        c.check()
        c.check_read([12])


def test_not_finite_rows_do_not_reach_their_block(dev):
    say("[cache8] not finite")

    def edit(kb, k, vb, v, first):
        f = first[0]
        for bits, x in ((kb, k), (vb, v)):
            bits[f + 1, 0, 5], x[f + 1, 0, 5] = 0x7F80, np.inf
            bits[f + 2, 0, 64:], x[f + 2, 0, 64:] = 0x7FC0, np.nan
            bits[f + 4, 0, 0], x[f + 4, 0, 0] = 0xFF80, -np.inf

    with np.errstate(invalid="ignore"):
        c = Cache8(dev, 1, 2, 1, 128, 16, 2, norm=False, rot=0, seed=8)
        c.append([0], [0], 0)
        c.append([1], [6], 6, edit=edit)
        c.check()
        c.append([4], [9], 9)
        c.check()
        c.check_read([14])


def test_pages_that_are_not_there(dev):
    """Rows on missing pages are dropped, queries come out all the same."""
    say("[cache8] missing pages")
    c = Cache8(dev, 2, 3, 2, 128, 16, 4, seed=9)
    t = c.ntable.copy()
    t[0, 1], t[1, 0] = -1, c.N
    before = c.pool.clone()
    c.append([0, 0], [40, 5], 40, table=torch.from_numpy(t).to(dev))
    hb = page_bytes8(2, 128, 16)
    got = c.pool.cpu().numpy().reshape(c.N, hb)
    want = np.full_like(got, 0xFF)
    full = np.full_like(got, 0xFF)
    OC.write_pages8(c.K[0], c.V[0], c.ntable[0], 16, full)
    for s in (0, 2):
        want[c.ntable[0, s]] = full[c.ntable[0, s]]
    written = ~np.all(got == before.cpu().numpy().reshape(c.N, hb), axis=1)
    assert set(np.flatnonzero(written)) == {int(c.ntable[0, 0]), int(c.ntable[0, 2])}
    zero = lambda x: np.where(x == 0x80, 0, x)      # a zero's sign is not compared
    assert np.array_equal(zero(got), zero(want))


def test_a_block_of_many_heads(dev):
    say("[cache8] 1024 heads")
    c = Cache8(dev, 1, 1024, 1024, 64, 16, 2, seed=10)
    c.append([0], [18], 18)
    c.check()


# ------------------------------------------------------------------ attention

class Case8(Case):
    """Case over 8-bit pages."""

    def __init__(self, dev, lens, ells, Hq, Hkv, D, P, gamma, window=0, sinks=0, packed=True, seed=1, peak=1.0,
                 max_pages=None, scale=None):
        rng = np.random.default_rng(seed)
        self.__dict__.update(fmt=FP8, lens=lens, ells=ells, Hq=Hq, Hkv=Hkv, D=D, P=P, gamma=gamma, window=window,
                             sinks=sinks, scale=D ** -0.5 if scale is None else scale, dev=dev)
        n = [min(max(e, -1), gamma) + 1 for e in ells]
        total = [a + b for a, b in zip(lens, n)]
        mp = max(1, max(-(-t // P) for t in total)) if max_pages is None else max_pages
        self.npool, self.ntable, self.ks, self.vs, self.held = build8(rng, total, Hkv, D, P, mp)
        first = (np.cumsum([0] + n)[:-1] + 1).tolist() if packed else [r * (gamma + 1) for r in range(len(lens))]
        self.rows = sum(n) + 2 if packed else len(lens) * (gamma + 1)
        self.first, self.n = first, n
        qb, self.nq = bf(rng.standard_normal((self.rows, Hq, D)) * peak)
        self.q = t16(qb, dev)
        self.row0 = i32(first, dev) if packed else None
        self.ell, self.length = i32(ells, dev), i32(lens, dev)
        self.pool, self.table = torch.from_numpy(self.npool).to(dev), torch.from_numpy(self.ntable).to(dev)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(x) for x in s))
def test_attention_against_oracle(shape, dev):
    say(f"[cache8] attention {shape}")
    lens, ells, Hq, Hkv, D, P, gamma, window, sinks, packed = shape
    Case8(dev, lens, ells, Hq, Hkv, D, P, gamma, window, sinks, packed).check()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_peaked_scores(D, dev):
    say(f"[cache8] peaked {D}")
    Case8(dev, [333, 40], [16, 2], 8, 2, D, 32, 16, peak=60.0, seed=4).check()
    Case8(dev, [333], [3], 8, 2, D, 32, 3, scale=0.0, seed=5).check()
    Case8(dev, [333], [3], 8, 2, D, 32, 3, scale=-0.2, seed=6).check()


def test_missing_pages_and_rows_that_see_nothing(dev):
    say("[cache8] attention, missing pages")
    for window, sinks in ((0, 0), (50, 20)):
        c = Case8(dev, [200, 90, 40, 10], [16, 3, 0, 5], 8, 2, 128, 16, 16, window, sinks)
        t = c.ntable.copy()
        t[0, 2:5] = -2
        t[1, 0] = t.max() + 100
        t[3, :] = -1
        c.table = torch.from_numpy(t).to(dev)
        have = []
        for r, k in enumerate(c.ks):
            j = np.arange(len(k)) // 16
            have.append((t[r, j] >= 0) & (t[r, j] < c.pool.shape[0]))
        c.check(have=have)


@pytest.mark.parametrize("D,rows", [(64, 16), (128, 16), (128, 0), (256, 5)])
def test_nan_values_reach_the_rows_that_see_them(D, rows, dev):
    """NaN codes among the last rows' values: rows before them are as without."""
    say(f"[cache8] NaN values {D} {rows}")
    c = Case8(dev, [70, 33], [rows, rows], 4, 2, D, 32, rows, seed=11)
    pool = c.npool.copy()
    hb = page_bytes8(1, D, 32)
    plain = torch.zeros((c.rows, 4, D), dtype=torch.bfloat16, device=dev)
    c.call(plain)
    want = np.zeros((c.rows, 4, D), bool)
    for r, (t, d) in enumerate(((70 + rows // 2, 3), (20, D - 1))):
        page = pool[c.ntable[r, t // 32]][:hb]                          # head 0
        v = page[32 * D + t % 32 // 16 * 16 * D:][:16 * D].reshape(2, 32, D // 32, 8)
        v[t % 16 // 8, d % 32, d // 32, t % 8] = 0xFF
        for i in range(c.n[r]):
            want[c.first[r] + i, :2, d] = c.lens[r] + i >= t
    c.pool = torch.from_numpy(pool).to(dev)
    out = torch.zeros_like(plain)
    c.call(out)
    assert np.array_equal(torch.isnan(out).cpu().numpy(), want)
    hide = torch.from_numpy(want).to(dev)
    assert torch.equal(out.masked_fill(hide, 0), plain.masked_fill(hide, 0))


def test_many_requests_and_far_pages(dev):
    """Offsets past 32 bits: the pool's pages lie beyond 4 GB."""
    say("[cache8] far pages")
    from semi_ar_draft_round_amd import binding as B
    H, D, P = 8, 128, 64
    nb = page_bytes8(H, D, P)
    N = 5_000_000_000 // nb
    c = Case8(dev, [100, 77], [3, 0], 16, H, D, P, 3, seed=12)
    pool = torch.empty((N, nb), dtype=torch.uint8, device=dev)
    used = c.ntable.max() + 1
    pool[N - used:] = c.pool[:used]
    near, far = (torch.zeros((c.rows, c.Hq, D), dtype=torch.bfloat16, device=dev) for _ in range(2))
    c.call(near)
    c.table = torch.where(c.table >= 0, c.table + (N - int(used)), c.table)
    c.pool = pool
    c.call(far)
    assert torch.equal(near, far)
    k0, v0 = B.dspark_cache_read(pool, c.table, None, c.length, 100, fmt=FP8, page=P, heads_kv=H, dim=D)
    assert np.array_equal(back(k0)[0], c.ks[0][:100]) and np.array_equal(back(v0)[1, :77], c.vs[1][:77])


def test_captured_and_on_another_stream(dev):
    """A captured append, attention and read, replayed between eager work on
    another stream: the eager results every time."""
    from semi_ar_draft_round_amd.cache import PagedCache
    say("[cache8] captured")
    g = torch.Generator().manual_seed(3)
    c = PagedCache(2, 3, 200, 24, 2, 128, page=16, fmt=FP8)
    ell = i32([5, 0, 3], dev)
    q, k, v = (torch.randn((18, h, 128), generator=g).to(torch.bfloat16).to(dev) for h in (4, 2, 2))
    out = torch.zeros_like(q)

    def step():
        c.reserve(ell, 5)
        for layer in range(2):
            o, _ = c.attend(layer, c.append(layer, q, k, v), out=out)
        c.commit(ell)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    c.reset()
    eager = []
    for _ in range(3):
        step()
        torch.cuda.synchronize()
        eager.append((out.clone(), c.length.clone(), c.read(1, 40)))
    c.reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    c.reset()
    for o, n, (rk, rv) in eager:
        graph.replay()
        torch.randn(1000, device=dev).sum()
        torch.cuda.synchronize()
        k1, v1 = c.read(1, 40)
        assert torch.equal(o[:6], out[:6]) and torch.equal(n, c.length) and torch.equal(rk, k1) and torch.equal(rv, v1)


def test_forked_blocks_and_moved_pages(dev):
    """A block that requests share and then go on with apart (its scales grow in
    the copies, not in the page the others read), and pages drawn together: as
    if every request had appended all of it itself."""
    from semi_ar_draft_round_amd.cache import PagedCache
    say("[cache8] forked")
    g = torch.Generator().manual_seed(11)
    D, n0, gamma = 64, 21, 24
    draw = lambda n, s: [(torch.randn((n, 2, D), generator=g) * s).to(torch.bfloat16).to(dev) for _ in range(2)]
    k0, v0 = draw(n0, 1.0)
    k1, v1 = draw(3 * (gamma + 1), 4000.0)
    q = torch.ones((3 * (gamma + 1), 2, D), dtype=torch.bfloat16, device=dev)
    forked, apart = (PagedCache(1, 3, 100, 14, 2, D, page=32, fmt=FP8) for _ in range(2))

    def append(c, ell, k, v):
        c.reserve(i32(ell, dev), gamma)
        assert c.ell.tolist() == ell
        c.append(0, q, k, v)
        c.commit(i32([max(e, 0) for e in ell], dev))

    def first(c, ell):
        k, v = (torch.zeros((3, gamma + 1, 2, D), dtype=torch.bfloat16, device=dev) for _ in range(2))
        k[:, :n0], v[:, :n0] = k0, v0
        append(c, ell, k.view(-1, 2, D), v.view(-1, 2, D))

    first(forked, [n0 - 1, -1, -1])
    first(apart, [n0 - 1] * 3)
    forked.fork(i32([0, 0, 0], dev))
    for c in (forked, apart):
        append(c, [0, 5, -1], k1, v1)
    k, v = forked.read(0, 60)
    assert all(torch.equal(a, b) for a, b in zip((k, v), apart.read(0, 60)))
    assert not torch.equal(k[0, :n0], k[2, :n0])          # the larger scale has cost slot 0's copy its small values
    for c in (forked, apart):
        append(c, [17, 24, 2], k1, v1)
        c.fork(i32([-1, 1, 2], dev))
        c.compact()
        append(c, [3, 0, 4], k1, v1)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(forked.read(0, 60), apart.read(0, 60)))
