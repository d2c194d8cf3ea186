"""dspark_cache_append and dspark_cache_read against the float64 oracle.

Tolerance of a normed and rotated 16-bit value y made of a pair (a, b): the
arithmetic is fp32 with at most 32 roundings on the way (a sum of D squares
over D / 8 lanes, a square root, a division, products, the rotation), each
2^-24 of |a| + |b|, doubled for the second-order terms; then one rounding to
bf16, half a step = 2^-8 of the value.  V bits and 4-bit values are exact
(keys of 4-bit pages are fp64 on both sides: a code may differ only where the
value is within 2^-40 of a border)."""

import sys

import numpy as np
import pytest

from cache_cases import BF16, F32, FP4, HALF, bf, page_bytes
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
    def __init__(self, rng, dev, fmt, lens, ells, Hq, Hkv, D, P, gamma, rot, adjacent, packed, dense, norms=True,
                 scale=1.0):
        R = len(lens)
        self.fmt, self.lens, self.ells, self.gamma, self.P, self.D, self.Hkv = fmt, lens, ells, gamma, P, D, Hkv
        n = [min(max(e, -1), gamma) + 1 for e in ells]
        if dense:
            self.row0, rows = None, R * (gamma + 1)
            first = [r * (gamma + 1) for r in range(R)]
        else:
            first = (np.cumsum([0] + n)[:-1] + 2).tolist()      # two rows in front belong to nobody
            rows = sum(n) + 4                                   # and two behind
            self.row0 = torch.tensor(first, dtype=torch.int32, device=dev)
        xb, x = bf(rng.standard_normal((rows, Hq + 2 * Hkv, D)) * scale)
        self.x, self.rows = x, rows
        xt = t16(xb, dev)
        q, k, v = xt[:, :Hq], xt[:, Hq:Hq + Hkv], xt[:, Hq + Hkv:]
        self.q, self.k, self.v = (q, k, v) if packed else (q.contiguous(), k.contiguous(), v.contiguous())
        wb, w = bf(1 + 0.4 * rng.standard_normal((2, D)))
        self.w = w if norms else [None, None]
        self.wq, self.wk = (t16(wb[0], dev), t16(wb[1], dev)) if norms else (None, None)
        self.freq = 1e4 ** (-2.0 * np.arange(rot // 2) / rot) if rot else None
        self.adjacent = adjacent
        mp = max(1, max(-(-(a + b) // P) for a, b in zip(lens, n)))
        need = [-(-(a + b) // P) for a, b in zip(lens, n)]
        ids = rng.permutation(sum(need) + 2)
        self.table = np.full((R, mp), -1, dtype=np.int32)
        at = 0
        for r, m in enumerate(need):
            self.table[r, :m] = ids[at:at + m]
            at += m
        self.pool0 = rng.integers(0, 256, (len(ids), page_bytes(fmt, Hkv, D, P))).astype(np.uint8)
        self.pool = torch.from_numpy(self.pool0.copy()).to(dev)
        self.ttable = torch.from_numpy(self.table).to(dev)
        self.ell = torch.tensor(ells, dtype=torch.int32, device=dev)
        self.length = torch.tensor(lens, dtype=torch.int32, device=dev)
        self.index = [(r, i, first[r] + i, lens[r] + i) for r in range(R) for i in range(n[r])]
        self.Hq = Hq

    def call(self, q_out=None):
        from semi_ar_draft_round_amd import binding as B
        return B.dspark_cache_append(self.q, self.k, self.v, self.pool, self.ttable, self.length, self.ell, self.gamma,
                                     fmt=self.fmt, page=self.P, wq=self.wq, wk=self.wk, eps=1e-5, adjacent=self.adjacent,
                                     freq=None if self.freq is None else torch.from_numpy(self.freq).to(self.pool.device),
                                     row0=self.row0, q_out=q_out)

    def want(self, sl, w):
        """The normed and rotated rows of heads sl, and the magnitude of each pair."""
        rows = [ix[2] for ix in self.index]
        pos = [ix[3] for ix in self.index]
        y = OC.norm(self.x[rows][:, sl], w, 1e-5)
        z = OC.rotate(y, pos, self.freq, self.adjacent)
        mag = np.abs(y)
        if self.freq is not None:
            one = OC.rotate(np.abs(y), np.zeros(len(pos)), self.freq, self.adjacent)
            h = len(self.freq)
            a = np.arange(h) * 2 if self.adjacent else np.arange(h)
            b = a + 1 if self.adjacent else a + h
            mag = one.copy()
            mag[..., a] = mag[..., b] = one[..., a] + one[..., b]
        return z, mag


CASES = [  # fmt, lens, ells, Hq, Hkv, D, P, gamma, rot, adjacent, packed, dense
    (1, [0], [0], 1, 1, 64, 16, 0, 64, False, False, True),
    (1, [1000003], [0], 4, 2, 128, 64, 0, 128, False, False, True),     # a far position
    (1, [5, 0, 17, 130], [16, -1, 3, 30], 14, 2, 128, 16, 16, 128, False, True, False),
    (1, [7, 8, 9, 15, 16], [0, 8, 9, 16, 15], 6, 3, 64, 32, 16, 32, True, True, True),
    (1, [3, 60], [70, 64], 8, 1, 256, 64, 70, 256, True, False, False),
    (1, [0, 33], [40, 7], 5, 5, 256, 128, 40, 128, False, True, False),
    (1, [2, 3], [4, 4], 2, 2, 128, 16, 4, 0, False, False, True),
    (2, [0], [0], 2, 1, 64, 16, 0, 64, False, False, True),
    (2, [5, 0, 17, 130], [16, -1, 3, 30], 14, 2, 128, 16, 16, 128, False, True, False),
    (2, [7, 8, 9, 15, 16, 1], [0, 8, 9, 16, 15, 4], 6, 3, 64, 32, 16, 32, True, True, True),
    (2, [3, 60], [70, 64], 8, 1, 256, 64, 70, 256, True, False, False),
    (2, [0, 33], [40, 7], 5, 5, 128, 128, 40, 0, False, True, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c))
def test_append_against_oracle(case, dev):
    from semi_ar_draft_round_amd import binding as B
    say(f"[append] {case}")
    far = case[1][0] > 100000
    rng = np.random.default_rng(7)
    if far:   # the page of the far position alone exists
        case = (*case[:1], [case[1][0] % case[6]], *case[2:])
    c = Case(rng, dev, *case)
    if far:
        shift = 1000003 // case[6] * case[6]
        c.length += shift
        wide = np.full((1, shift // case[6] + 1), -1, dtype=np.int32)
        wide[0, -1] = c.table[0, 0]
        c.ttable = torch.from_numpy(wide).to(dev)
        c.index = [(r, i, row, p + shift) for r, i, row, p in c.index]
    q_out = torch.full((c.rows, c.Hq, c.D), 7.0, dtype=torch.bfloat16, device=dev)
    c.call(q_out)
    torch.cuda.synchronize()
    rows = [ix[2] for ix in c.index]
    got = back(q_out)
    z, mag = c.want(slice(0, c.Hq), c.w[0])
    assert np.all(np.abs(got[rows] - z) <= HALF * np.abs(z) + 64 * F32 * mag)
    left = np.ones(c.rows, dtype=bool)
    left[rows] = False
    assert np.all(got[left] == 7.0)              # rows of nobody are as they were

    # the pages: exactly what the layout says, every other byte as it was
    T = c.gamma + 1
    start = c.length
    count = torch.tensor([min(max(e, -1), c.gamma) + 1 for e in c.ells], dtype=torch.int32, device=dev)
    k = torch.full((len(c.lens), T, c.Hkv, c.D), 3.0, dtype=torch.bfloat16, device=dev)
    v = k.clone()
    B.dspark_cache_read(c.pool, c.ttable, start, count, T, fmt=c.fmt, page=c.P, heads_kv=c.Hkv, dim=c.D, k=k, v=v)
    torch.cuda.synchronize()
    kd, vd = back(k), back(v)
    at = ([ix[0] for ix in c.index], [ix[1] for ix in c.index])
    z, mag = c.want(slice(c.Hq, c.Hq + c.Hkv), c.w[1])
    val = c.x[rows][:, c.Hq + c.Hkv:]
    if c.fmt == BF16:
        assert np.all(np.abs(kd[at] - z) <= HALF * np.abs(z) + 64 * F32 * mag)
        assert np.array_equal(vd[at], val)
    else:
        want = OC.quantise_k(z)
        g = np.abs(z.reshape(*z.shape[:-1], -1, 32))
        border = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0])
        e = np.exp2(np.floor(np.log2(g.max(-1, keepdims=True))) - 2)
        near = (np.abs(g[..., None] / e[..., None] - np.concatenate([border, 2 * border])) < 2.0 ** -40).any(-1)
        ok = (kd[at] == want) | near.any(-1, keepdims=True).repeat(32, -1).reshape(z.shape)
        assert ok.all()
        assert near.mean() < 1e-3
        q4 = OC.quantise_v(val)
        # the product of a code and the fp32 scale, rounded to bf16
        assert np.all(np.abs(vd[at] - q4) <= HALF * np.abs(q4) * (1 + HALF))
    gone = np.ones(kd.shape[:2], dtype=bool)
    gone[at] = False
    assert np.all(kd[gone] == 3.0) and np.all(vd[gone] == 3.0)

    # bytes outside the new tokens are untouched: read every older token before and after
    old = torch.from_numpy(c.pool0).to(dev)
    used = set()
    for r, i, _, p in c.index:
        used.add((int(c.ttable[r, p // c.P]), p % c.P))
    n_pages = old.shape[0]
    whole = torch.arange(n_pages, dtype=torch.int32, device=dev).view(n_pages, 1)
    full = torch.full((n_pages,), c.P, dtype=torch.int32, device=dev)
    a = B.dspark_cache_read(old, whole, None, full, c.P, fmt=c.fmt, page=c.P, heads_kv=c.Hkv, dim=c.D)
    b = B.dspark_cache_read(c.pool, whole, None, full, c.P, fmt=c.fmt, page=c.P, heads_kv=c.Hkv, dim=c.D)
    keep = torch.ones(n_pages, c.P, dtype=torch.bool)
    for page, t in used:
        keep[page, t] = False
    for x, y in zip(a, b):
        assert torch.equal(x.cpu().view(torch.int16)[keep], y.cpu().view(torch.int16)[keep])
    if c.fmt == BF16:
        assert int((old != c.pool).any(dim=1).sum()) <= len({p for p, _ in used})


def test_read_agrees_with_the_written_layout(dev):
    """Pages written by the oracle's layout, read by the library."""
    from cache_cases import build
    from semi_ar_draft_round_amd import binding as B
    for fmt in (BF16, FP4):
        for D, P, H in ((64, 16, 3), (128, 64, 2), (256, 32, 1)):
            say(f"[read] {fmt} {D} {P}")
            rng = np.random.default_rng(D + P)
            lens = [75, 1, 0, 40]
            pool, table, ks, vs = build(rng, fmt, lens, H, D, P, 6)
            start = torch.tensor([3, 0, 0, 8], dtype=torch.int32, device=dev)
            count = torch.tensor([72, 1, 0, 9], dtype=torch.int32, device=dev)
            k, v = B.dspark_cache_read(torch.from_numpy(pool).to(dev), torch.from_numpy(table).to(dev), start, count, 80,
                                       fmt=fmt, page=P, heads_kv=H, dim=D)
            torch.cuda.synchronize()
            kd, vd = back(k), back(v)
            for r, (s, n) in enumerate(zip([3, 0, 0, 8], [72, 1, 0, 9])):
                assert np.array_equal(kd[r, :n], ks[r][s:s + n])
                assert np.all(np.abs(vd[r, :n] - vs[r][s:s + n]) <= (0 if fmt == BF16 else HALF * 1.01) * np.abs(vs[r][s:s + n]))
                assert not kd[r, n:].any() and not vd[r, n:].any()
            # no page: zeros; a count past T: T rows
            hole = torch.from_numpy(table).to(dev)
            hole[0, 1] = -1
            hole[3, 0] = 10 ** 6
            k, _ = B.dspark_cache_read(torch.from_numpy(pool).to(dev), hole, None, count + 1000, 70, fmt=fmt, page=P,
                                       heads_kv=H, dim=D)
            kd = back(k)
            lo, hi = P, min(2 * P, 70)
            assert not kd[0, lo:hi].any() and not kd[3, :min(P, 70)].any()
            assert np.array_equal(kd[0, :lo], ks[0][:lo])


def test_special_values(dev):
    """Zero heads, infinities, NaNs and the largest and smallest values."""
    from semi_ar_draft_round_amd import binding as B
    rng = np.random.default_rng(3)
    for fmt in (BF16, FP4):
        c = Case(rng, dev, fmt, [3], [15], 2, 2, 64, 16, 15, 0, False, False, True, norms=False)
        x = c.k.clone()
        x[0] = 0
        x[1, 0, 5] = float("inf")
        x[2, 1, 40] = float("nan")
        x[3] = 3.3e38
        x[4] = 1e-38
        c.k = x
        c.v = x.clone()
        c.call()
        count = torch.tensor([16], dtype=torch.int32, device=dev)
        k, v = B.dspark_cache_read(c.pool, c.ttable, c.length, count, 16, fmt=fmt, page=16, heads_kv=2, dim=64)
        xs, kd, vd = back(x), back(k)[0], back(v)[0]
        if fmt == BF16:
            assert np.array_equal(kd, xs, equal_nan=True) and np.array_equal(vd, xs, equal_nan=True)
            continue
        assert not kd[0].any() and not vd[0].any()
        # an infinity or a NaN makes its scale group NaN: 32 dims of K, the head of V
        assert np.isnan(kd[1, 0, :32]).all() and np.isfinite(kd[1, 0, 32:]).all() and np.isfinite(kd[1, 1]).all()
        assert np.isnan(kd[2, 1, 32:]).all() and np.isfinite(kd[2, 1, :32]).all()
        assert np.isnan(vd[1, 0]).all() and np.isfinite(vd[1, 1]).all() and np.isnan(vd[2, 1]).all()
        assert np.all(np.abs(kd[3] - xs[3]) <= xs[3] / 4) and np.all(np.abs(vd[3] / xs[3] - 1) <= 2 * HALF)
        assert np.all(np.abs(kd[4] - xs[4]) <= 2.0 ** -126) and np.all(np.isfinite(vd[4]))


def test_other_stream_graph_and_repeat(dev):
    """On a side stream, captured and replayed between eager work, and twice:
    the same bits every time."""
    for fmt in (BF16, FP4):
        c = Case(np.random.default_rng(5), dev, fmt, [9, 30, 2], [16, 3, 8], 8, 2, 128, 32, 16, 128, False, True, False)
        q0 = torch.zeros((c.rows, c.Hq, c.D), dtype=torch.bfloat16, device=dev)
        c.freq_t = torch.from_numpy(c.freq).to(dev)
        from semi_ar_draft_round_amd import binding as B

        def go(q_out):
            B.dspark_cache_append(c.q, c.k, c.v, c.pool, c.ttable, c.length, c.ell, c.gamma, fmt=fmt, page=c.P, wq=c.wq,
                                  wk=c.wk, freq=c.freq_t, row0=c.row0, q_out=q_out)
        go(q0)
        torch.cuda.synchronize()
        pool = c.pool.clone()
        first = torch.from_numpy(c.pool0).to(dev)
        side = torch.cuda.Stream()
        c.pool.copy_(first)
        q1 = torch.zeros_like(q0)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            go(q1)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(q0, q1) and torch.equal(pool, c.pool)
        g = torch.cuda.CUDAGraph()
        q2 = torch.zeros_like(q0)
        with torch.cuda.graph(g):
            go(q2)
        for _ in range(4):
            c.pool.copy_(first)
            q2.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(q0, q2) and torch.equal(pool, c.pool)


def test_no_rows(dev):
    from semi_ar_draft_round_amd import binding as B
    e = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=dev)
    i = lambda *s: torch.full(s, -1, dtype=torch.int32, device=dev)
    pool = torch.zeros(2, B.dspark_cache_page_bytes(1, 2, 64, 16), dtype=torch.uint8, device=dev)
    out = B.dspark_cache_append(e(0, 4, 64), e(0, 2, 64), e(0, 2, 64), pool, i(3, 2), i(3) + 1, i(3), 5, fmt=1, page=16,
                                row0=i(3) + 1)
    assert out.shape == (0, 4, 64)
