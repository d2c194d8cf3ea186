"""dspark_cache_weigh against the float64 oracle, over pages of all formats.

Bound of a weight's error: a score is an fp32 sum of D exact products and a few
scalings, off by at most (D + 8) 2^-24 of the sum of magnitudes; the log-sum is
given, its product with log2 e off by 2^-23 of it; the exponential as much in
relative terms (e^x - 1 < 2 x) and 2^-22 itself.  The sum over N weights is
fp32, in any order: N + 64 roundings of 2^-24."""

import sys

import numpy as np
import pytest

from cache8_cases import FP8, build8
from cache_cases import BF16, F32, FP4, bf, build
from oracle import cache as OC
from test_gpu_cache_attention import SHAPES, t16

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


class Case:
    def __init__(self, dev, fmt, lens, ells, Hq, Hkv, D, P, gamma, window=0, sinks=0, packed=True, seed=1, peak=1.0,
                 scale=None, more=2, drop=None):
        rng = np.random.default_rng(seed)
        self.__dict__.update(fmt=fmt, lens=lens, ells=ells, Hq=Hq, Hkv=Hkv, D=D, P=P, gamma=gamma, window=window,
                             sinks=sinks, scale=D ** -0.5 if scale is None else scale, dev=dev)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
        n = [min(max(e, -1), gamma) + 1 for e in ells]
        total = [max(a, 0) + b for a, b in zip(lens, n)]
        mp = max(1, max(-(-t // P) for t in total)) + more
        made = build8(rng, total, Hkv, D, P, mp) if fmt == FP8 else build(rng, fmt, total, Hkv, D, P, mp)
        self.npool, self.ntable, self.ks = made[0], made[1], made[2]
        if drop:
            drop(self.ntable)
        self.first = (np.cumsum([0] + n)[:-1] + 1).tolist() if packed else [r * (gamma + 1) for r in range(len(lens))]
        self.rows, self.n = sum(n) + 2 if packed else len(lens) * (gamma + 1), n
        qb, self.nq = bf(rng.standard_normal((self.rows, Hq, D)) * peak)
        self.q, self.row0 = t16(qb, dev), i32(self.first) if packed else None
        self.ell, self.length = i32(ells), i32(lens)
        self.pool, self.table = torch.from_numpy(self.npool).to(dev), torch.from_numpy(self.ntable).to(dev)
        self.have, self.nlse = [], np.full((self.rows, Hq), np.nan, np.float32)
        for r, (f, m) in enumerate(zip(self.first, n)):
            ids = self.ntable[r, np.arange(total[r]) // P]
            self.have.append((ids >= 0) & (ids < len(self.npool)))
            if m and lens[r] >= 0:
                _, z = OC.attention(self.nq[f:f + m], self.ks[r], self.ks[r], lens[r] + np.arange(m), self.scale, window,
                                    sinks, self.have[r])
                self.nlse[f:f + m] = z
        self.lse = torch.from_numpy(self.nlse).to(dev)
        self.old = rng.uniform(0, 4, (len(lens), mp)).astype(np.float32)

    def call(self, keep, mass, **kw):
        from semi_ar_draft_round_amd import binding as B
        B.dspark_cache_weigh(self.q, kw.pop("lse", self.lse), self.pool, self.table, self.length, self.ell, self.gamma,
                             mass, keep=keep, fmt=self.fmt, page=self.P, heads_kv=self.Hkv, scale=self.scale,
                             window=self.window, sinks=self.sinks, row0=self.row0, **kw)
        torch.cuda.synchronize()
        return mass.cpu().numpy().astype(np.float64)

    def check(self, keep=1.0):
        got = self.call(keep, torch.from_numpy(self.old.copy()).to(self.dev))
        worst = 0.0
        for r, (f, m) in enumerate(zip(self.first, self.n)):
            if m == 0 or self.lens[r] < 0:
                assert np.array_equal(got[r], self.old[r].astype(np.float64))
                continue
            q, z, pos = self.nq[f:f + m], self.nlse[f:f + m], self.lens[r] + np.arange(m)
            w = OC.weigh(q, z, self.ks[r], pos, self.scale, self.window, self.sinks, self.P, self.have[r])
            want = np.float64(np.float32(keep)) * self.old[r].astype(np.float64)
            want[:len(w)] += w
            ka = np.nan_to_num(np.abs(self.ks[r]), nan=0.0).max(0)
            mag = (np.abs(q) * np.repeat(ka, self.Hq // self.Hkv, axis=0)[None]).sum(-1) * abs(self.scale)
            zz = np.where(np.isfinite(z), np.abs(z), 0)
            rel = 2 * ((self.D + 8) * F32 * mag + 2.0 ** -23 * zz).max() + 2.0 ** -22 + (m * self.Hq * self.P + 64) * F32
            tol = rel * want + 1e-30
            assert np.all(np.abs(got[r] - want) <= tol), (r, float((np.abs(got[r] - want) / tol).max()))
            worst = max(worst, float((np.abs(got[r] - want) / tol).max()))
        say(f"  worst error {worst:.3f} of its bound")
        return got


@pytest.mark.parametrize("fmt", [BF16, FP4, FP8])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(x) for x in s))
def test_weigh_against_oracle(shape, fmt, dev):
    say(f"[weigh] fmt {fmt} {shape}")
    lens, ells, Hq, Hkv, D, P, gamma, window, sinks, packed = shape
    c = Case(dev, fmt, lens, ells, Hq, Hkv, D, P, gamma, window, sinks, packed)
    c.check()
    c.check(keep=0.5)


@pytest.mark.parametrize("fmt", [BF16, FP4, FP8])
def test_every_row_and_head_shares_out_one(fmt, dev):
    say(f"[weigh] sums {fmt}")
    c = Case(dev, fmt, [500, 40], [16, 3], 8, 2, 128, 32, 16, seed=2)
    got = c.call(0.0, torch.from_numpy(c.old).to(dev))
    for r, m in enumerate(c.n):
        assert abs(got[r].sum() - m * 8) < 1e-3 * m * 8


@pytest.mark.parametrize("fmt", [BF16, FP8])
def test_missing_pages_and_rows_that_see_nothing(fmt, dev):
    say(f"[weigh] missing pages {fmt}")

    def drop(t):
        t[0, 2:5] = -2
        t[1, 0] = 1 << 29
        t[3, :] = -1

    for window, sinks in ((0, 0), (50, 20)):
        for P in (16, 64):
            Case(dev, fmt, [200, 90, 40, 10], [16, 3, 0, 5], 8, 2, 128, P, 16, window, sinks, drop=drop).check(keep=0.25)


@pytest.mark.parametrize("fmt", [BF16, FP4, FP8])
def test_peaked_scores(fmt, dev):
    say(f"[weigh] peaked {fmt}")
    Case(dev, fmt, [333, 40], [16, 2], 8, 2, 64, 32, 16, peak=40.0, seed=4).check()
    Case(dev, fmt, [333], [3], 8, 2, 128, 16, 3, scale=0.0, seed=5).check()
    Case(dev, fmt, [333], [3], 8, 2, 256, 32, 3, scale=-0.2, seed=6).check()


def test_many_slots(dev):
    """More slots than threads, most of them idle, lengths of every kind; and a
    long context beside short ones, under a window."""
    say("[weigh] slots")
    rng = np.random.default_rng(7)
    R = 700
    lens = [int(x) for x in rng.integers(0, 120, R)]
    ells = [int(x) if rng.random() < 0.1 else -1 for x in rng.integers(0, 5, R)]
    ells[699], lens[3], ells[5], lens[5] = 4, -1, 2, 0
    Case(dev, BF16, lens, ells, 4, 2, 64, 16, 4, seed=8).check(keep=0.5)
    Case(dev, FP8, [9000, 3, 700], [2, 0, 1], 4, 2, 64, 16, 2, window=300, sinks=40, seed=9).check(keep=0.5)


def test_nan_stays_where_it_is_seen(dev):
    """A NaN key makes its page's mass NaN and no other's; a NaN log-sum those
    of the pages its row sees; what lies behind the rows does nothing."""
    say("[weigh] NaN")
    c = Case(dev, BF16, [100], [0], 2, 1, 64, 16, 0, window=40, sinks=0, packed=False, seed=10)
    half = c.pool.clone()
    page = half[int(c.ntable[0, 4])].view(torch.bfloat16)
    page[:64] = float("nan")
    c.pool = half
    got = c.call(1.0, torch.from_numpy(c.old.copy()).to(dev))
    assert np.isnan(got[0, 4]) and np.isfinite(np.delete(got[0], 4)).all()
    c = Case(dev, BF16, [100], [1], 2, 1, 64, 16, 1, window=40, sinks=0, packed=False, seed=10)
    lse = c.lse.clone()
    lse[1, 0] = float("nan")
    got = c.call(1.0, torch.from_numpy(c.old.copy()).to(dev), lse=lse)
    seen = [s for s in range(c.old.shape[1]) if s * 16 <= 101 and s * 16 + 15 > 101 - 40]
    assert np.isnan(got[0, seen]).all() and np.isfinite(np.delete(got[0], seen)).all()


def test_repeated_captured_and_on_another_stream(dev):
    say("[weigh] captured")
    c = Case(dev, FP8, [900, 64, 333], [16, 3, 9], 14, 2, 128, 64, 16, seed=11)
    first = torch.from_numpy(c.old).to(dev)
    a = torch.from_numpy(c.call(0.5, first.clone())).clone()
    assert torch.equal(a, torch.from_numpy(c.call(0.5, first.clone())))
    mass = first.clone()
    from semi_ar_draft_round_amd import binding as B
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    args = dict(keep=0.5, fmt=c.fmt, page=c.P, heads_kv=c.Hkv, scale=c.scale, row0=c.row0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        B.dspark_cache_weigh(c.q, c.lse, c.pool, c.table, c.length, c.ell, c.gamma, mass, **args)
    for _ in range(4):
        mass.copy_(first)
        g.replay()
        torch.randn(1000, device=dev).sum()
        torch.cuda.synchronize()
        assert torch.equal(a, mass.cpu().double())


def test_far_pages(dev):
    """Keys beyond 4 GB of the pool."""
    say("[weigh] far pages")
    for fmt in (BF16, FP8):
        c = Case(dev, fmt, [100, 77], [3, 0], 16, 8, 128, 64, 3, seed=12)
        near = c.call(0.0, torch.from_numpy(c.old).to(dev))
        nb = c.npool.shape[1]
        N = 5_000_000_000 // nb
        pool = torch.empty((N, nb), dtype=torch.uint8, device=dev)
        used = int(c.ntable.max()) + 1
        pool[N - used:] = c.pool[:used]
        c.pool, c.table = pool, torch.where(c.table >= 0, c.table + (N - used), c.table)
        assert np.array_equal(near, c.call(0.0, torch.from_numpy(c.old).to(dev)))
        del pool
        c.pool = None
