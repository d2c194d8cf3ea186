"""dspark_cache_evict against the oracle, bit for bit, and what the other calls
make of tables with evicted pages."""

import sys

import numpy as np
import pytest

from oracle import cache as OC

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


class State:
    """The oracle's pages on the device."""

    def __init__(self, pages, dev):
        self.o, self.dev = pages, dev
        i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(dev)
        self.table, self.len, self.ref = i32(pages.table), i32(pages.len), i32(pages.refs())
        self.bits = i32(self.words(pages.refs()))

    def words(self, ref):
        n = -(-len(ref) // 32)
        free = np.zeros(n * 32, bool)
        free[:len(ref)] = ref == 0
        return np.packbits(free.reshape(n, 32), axis=1, bitorder="little").view(np.uint32)[:, 0].view(np.int32)

    def four(self):
        return self.table, self.len, self.ref, self.bits

    def check(self):
        torch.cuda.synchronize()
        assert np.array_equal(self.table.cpu().numpy(), self.o.table)
        assert np.array_equal(self.len.cpu().numpy(), self.o.len)
        ref = self.o.refs()
        assert np.array_equal(self.ref.cpu().numpy(), ref)
        assert np.array_equal(self.bits.cpu().numpy(), self.words(ref))

    def evict(self, mass, budget, sinks, recent):
        from semi_ar_draft_round_amd import binding as B
        m = torch.from_numpy(mass.copy()).to(self.dev)
        b = torch.tensor(budget, dtype=torch.int32, device=self.dev)
        freed = B.dspark_cache_evict(*self.four(), m, b, page=self.o.P, sinks=sinks, recent=recent)
        want = mass.copy()
        gone = self.o.evict(want, budget, sinks, recent)
        self.check()
        assert freed.tolist() == gone
        assert np.array_equal(m.cpu().numpy().view(np.int32), want.view(np.int32))
        return gone


def filled(rng, lens, P, max_pages, spare=5, shared=()):
    """Requests with pages for their tokens; (r, s, n): r's first n pages are s's."""
    need = [-(-max(n, 0) // P) for n in lens]
    p = OC.Pages(len(lens), sum(need) + spare, max_pages, P)
    ids = rng.permutation(p.N)
    at = 0
    for r, n in enumerate(need):
        p.table[r, :n] = ids[at:at + n]
        at += n
        p.len[r] = lens[r]
    for r, s, n in shared:
        p.table[r, :n] = p.table[s, :n]
    return p


def weights(rng, shape, kind):
    m = rng.gamma(0.3, 5.0, shape).astype(np.float32)
    if kind == "ties":
        m = np.round(m).astype(np.float32)
        m[rng.random(shape) < 0.2] = -0.0
    if kind == "odd":
        m[rng.random(shape) < 0.1] = np.nan
        m[rng.random(shape) < 0.1] = np.inf
        m[rng.random(shape) < 0.1] = -np.inf
        m[rng.random(shape) < 0.1] = -m[0, 0] - 1
        m[rng.random(shape) < 0.1] = 1e-42          # subnormal
    return m


@pytest.mark.parametrize("kind", ["plain", "ties", "odd"])
@pytest.mark.parametrize("P,sinks,recent", [(16, 0, 0), (16, 1, 1), (32, 33, 100), (64, 64, 64), (128, 0, 1 << 30),
                                            (16, 2 ** 31 - 1, 2 ** 31 - 1)])
def test_evict_against_oracle(P, sinks, recent, kind, dev):
    say(f"[evict] {P} {sinks} {recent} {kind}")
    rng = np.random.default_rng(P + len(kind))
    lens = [0, 1, P, 7 * P + 3, 300 * P, 299 * P + 1, 40 * P, 40 * P, -1, 12 * P]
    p = filled(rng, lens, P, 301, shared=((7, 6, 25), (9, 4, 12)))
    s = State(p, dev)
    for budget in ([3] * 10, [0, 0, 0, -1, 290, 1, 30, 20, 0, 5], [0] * 10, [2 ** 31 - 1] * 10):
        s.evict(weights(rng, p.table.shape, kind), budget, sinks, recent)


def test_long_tables(dev):
    """Tables past what a thread keeps in registers or a work group of either
    size takes, and whose length is just that."""
    say("[evict] long tables")
    rng = np.random.default_rng(3)
    for M, lens in ((512, [16 * 512, 16 * 500 - 5]), (513, [16 * 513, 16 * 300]), (1025, [16 * 1025, 16]), (8192, [16 * 8192, 16 * 8000 - 5]), (8193, [16 * 8193, 16 * 3]), (30000, [16 * 30000 - 9, 16 * 29000])):
        p = filled(rng, lens, 16, M)
        s = State(p, dev)
        for kind, budget in (("ties", [M // 2, 2]), ("odd", [100, 7]), ("plain", [0, 0])):
            s.evict(weights(rng, p.table.shape, kind), budget, 4, 50)


def test_all_alike_go_from_the_front(dev):
    say("[evict] all alike")
    p = filled(np.random.default_rng(4), [16 * 3000], 16, 3000)
    s = State(p, dev)
    assert s.evict(np.zeros((1, 3000), np.float32), [1000], 16, 0) == [2000]
    assert np.all(p.table[0, 1:2001] == -2) and p.table[0, 0] >= 0 and np.all(p.table[0, 2001:] >= 0)


def test_commit_under_a_window_takes_what_eviction_left(dev):
    """The window's release looks for pages from the back: it must not stop at
    an evicted one."""
    from semi_ar_draft_round_amd import binding as B
    say("[evict] window")
    rng = np.random.default_rng(5)
    p = filled(rng, [16 * 400, 16 * 400, 16 * 100], 16, 500)
    s = State(p, dev)
    m = weights(rng, p.table.shape, "plain")
    m[1, 60:330] = 0                                   # a run of evicted pages longer than a wave
    s.evict(m, [150, 130, 99], 20, 40)
    for window in (700, 300):
        ell = [4, 4, -1]
        out, pairs, refused = p.reserve(ell, 4)
        assert not refused and not pairs
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
        got, _, _, _ = B.dspark_cache_reserve(*s.four(), i32(ell), 4, page=16)
        s.check()
        B.dspark_cache_commit(*s.four(), got, i32([2, 4, 0]), 4, page=16, window=window, sinks=20)
        p.commit(out, [2, 4, 0], 4, window, 20)
        s.check()


@pytest.mark.parametrize("M", [40, 3000])
def test_fork_reserve_and_compact_after_eviction(M, dev):
    """Marks of evicted pages go with a fork, and pages that come back are the
    next to be handed out."""
    from semi_ar_draft_round_amd import binding as B
    say(f"[evict] fork {M}")
    rng = np.random.default_rng(6)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    lens = [16 * 37 + 3, 16 * 20, 5, 16 * 30]
    p = filled(rng, lens, 16, M, spare=2)
    s = State(p, dev)
    s.evict(weights(rng, p.table.shape, "plain"), [9, 20, 1, 3], 0, 16)
    parent = [0, 0, 3, 3]
    B.dspark_cache_fork(*s.four(), i32(parent), page=16)
    p.fork(parent)
    s.check()
    assert (p.table[1] == -2).sum() == (p.table[0] == -2).sum() > 0
    s.evict(weights(rng, p.table.shape, "plain"), [8, 4, 3, 2], 0, 0)      # shared ones stay the others'
    ell = [20, 0, 3, -1]
    out, pairs, _ = p.reserve(ell, 20)
    got, gpairs, n, _ = B.dspark_cache_reserve(*s.four(), i32(ell), 20, page=16)
    s.check()
    assert got.tolist() == out and gpairs[:int(n)].tolist() == [list(x) for x in pairs]
    moves = p.compact()
    gpairs, n = B.dspark_cache_compact(s.table, s.ref, s.bits)
    s.check()
    assert gpairs[:int(n)].tolist() == [list(x) for x in moves]


def test_captured_and_replayed(dev):
    from semi_ar_draft_round_amd import binding as B
    say("[evict] captured")
    rng = np.random.default_rng(7)
    p = filled(rng, [16 * 200, 16 * 150], 16, 200, shared=((1, 0, 30),))
    s = State(p, dev)
    mass = torch.from_numpy(weights(rng, p.table.shape, "ties")).to(dev)
    budget, freed = torch.tensor([50, 20], dtype=torch.int32, device=dev), torch.zeros(2, dtype=torch.int32, device=dev)
    start = [t.clone() for t in (*s.four(), mass)]
    B.dspark_cache_evict(*s.four(), mass, budget, page=16, sinks=4, recent=20, freed=freed)
    torch.cuda.synchronize()
    want = [t.clone() for t in (*s.four(), mass, freed)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.dspark_cache_evict(*s.four(), mass, budget, page=16, sinks=4, recent=20, freed=freed)
    for _ in range(4):
        for t, x in zip((*s.four(), mass), start):
            t.copy_(x)
        g.replay()
        torch.randn(1000, device=dev).sum()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*s.four(), mass, freed), want))
