"""The cache's page calls (dspark_cache_reset, reserve, commit, fork, compact,
copy) against the oracle's one-request-at-a-time bookkeeping: all integers,
equal exactly."""

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


class Both:
    """The oracle's pages and the device's, stepped together."""

    def __init__(self, R, n_pages, max_pages, P, dev):
        from semi_ar_draft_round_amd import binding as B
        self.B, self.P, self.dev = B, P, dev
        self.o = OC.Pages(R, n_pages, max_pages, P)
        i32 = dict(dtype=torch.int32, device=dev)
        self.table = torch.full((R, max_pages), 77, **i32)
        self.length, self.ref = torch.full((R,), 5, **i32), torch.full((n_pages,), 9, **i32)
        self.bits = torch.full(((n_pages + 31) // 32,), 3, **i32)
        B.dspark_cache_reset(self.table, self.length, self.ref, self.bits)
        self.same()

    @property
    def state(self):
        return self.table, self.length, self.ref, self.bits

    def i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device=self.dev)

    def same(self):
        torch.cuda.synchronize()
        o, ref = self.o, self.o.refs()
        assert np.array_equal(self.table.cpu().numpy(), o.table)
        assert np.array_equal(self.length.cpu().numpy(), o.len)
        assert np.array_equal(self.ref.cpu().numpy(), ref)
        words = np.zeros(self.bits.numel() * 32, dtype=bool)
        words[:o.N] = ref == 0
        got = np.unpackbits(self.bits.cpu().numpy().view(np.uint8), bitorder="little").astype(bool)
        assert np.array_equal(got, words)

    def reserve(self, ell, gamma):
        want, pairs, refused = self.o.reserve(ell, gamma)
        e, p, n, st = self.B.dspark_cache_reserve(*self.state, self.i32(ell), gamma, page=self.P)
        torch.cuda.synchronize()
        assert e.tolist() == want
        assert int(n) == len(pairs) and p[:len(pairs)].tolist() == [list(x) for x in pairs]
        assert int(st) == (self.B.ENOPAGES if refused else 0)
        self.same()
        return want

    def commit(self, ell, n_acc, gamma, window=0, sinks=0):
        self.o.commit(ell, n_acc, gamma, window, sinks)
        self.B.dspark_cache_commit(*self.state, self.i32(ell), self.i32(n_acc), gamma, page=self.P, window=window,
                                   sinks=sinks)
        self.same()

    def fork(self, parent):
        self.o.fork(parent)
        self.B.dspark_cache_fork(*self.state, self.i32(parent), page=self.P)
        self.same()

    def compact(self):
        want = self.o.compact()
        p, n = self.B.dspark_cache_compact(self.table, self.ref, self.bits)
        torch.cuda.synchronize()
        assert int(n) == len(want) and p[:len(want)].tolist() == [list(x) for x in want]
        self.same()


@pytest.mark.parametrize("R,n_pages,max_pages,P,gamma,window,sinks",
                         [(1, 1, 1, 16, 0, 0, 0), (3, 20, 5, 16, 4, 0, 0), (17, 90, 6, 16, 16, 40, 5),
                          (64, 333, 9, 32, 16, 33, 40), (130, 1000, 30, 16, 64, 100, 16), (5, 40, 9, 128, 200, 1, 0)])
def test_random_rounds(R, n_pages, max_pages, P, gamma, window, sinks, dev):
    """Rounds of fork, reserve (running out of pages now and then), commit and
    compact, with out-of-range ell, n_acc and parents among them."""
    rng = np.random.default_rng(R * 1000 + n_pages)
    b = Both(R, n_pages, max_pages, P, dev)
    for step in range(25):
        say(f"[pages] R {R} pages {n_pages} step {step}")
        if step % 3 == 2:
            parent = np.arange(R)
            pick = rng.random(R) < 0.3
            parent[pick] = rng.integers(-3, R + 2, pick.sum())
            b.fork(parent.tolist())
        ell = rng.integers(-2, gamma + 3, R).tolist()
        got = b.reserve(ell, gamma)
        if step % 5 == 1:
            got = b.reserve(got, gamma)        # again: everything is there already
        b.commit(got, rng.integers(-1, gamma + 2, R).tolist(), gamma, window, sinks)
        if step % 7 == 3:
            b.compact()
        if step % 6 == 5:                      # let a third of the requests go
            b.fork([r if rng.random() < 0.67 else -1 for r in range(R)])


def test_permutation_and_swap(dev):
    b = Both(6, 60, 6, 16, dev)
    b.commit(b.reserve([3, 20, 40, 0, 17, 60], 63), [2, 20, 11, 0, 16, 60], 63)
    b.fork([1, 0, 3, 4, 5, 2])                 # swaps and a cycle
    b.fork([0, 0, 0, 0, 0, 0])
    b.fork([-1] * 6)
    assert int(b.ref.sum()) == 0


def test_shared_tail_of_many_holders(dev):
    """Nine holders of one partly filled page, some of them writing: all but
    the last writer copy, and with too few pages the ones refused keep theirs
    untouched."""
    for n_pages in (64, 12, 6, 4):
        b = Both(9, n_pages, 4, 16, dev)
        b.commit(b.reserve([4] + [-1] * 8, 4), [4] + [0] * 8, 4)
        b.fork([0] * 9)
        ell = b.reserve([0, -1, 1, 2, 3, 4, -1, 14, 20], 20)
        b.commit(ell, [0] * 9, 20)
        b.reserve([0] * 9, 20)


def test_many_requests_and_a_large_pool(dev):
    """The largest batch, on a pool whose bitmap has many words per thread."""
    rng = np.random.default_rng(8)
    R = 4096
    b = Both(R, 100_001, 16, 16, dev)
    for step in range(2):
        say(f"[pages] many {step}")
        ell = rng.integers(-1, 40, R).tolist()
        b.commit(b.reserve(ell, 39), rng.integers(0, 40, R).tolist(), 39)
        b.fork([r if r % 5 else (r + 1) % R for r in range(R)])
    b.compact()


def test_copy_moves_pages_of_every_layer(dev):
    from semi_ar_draft_round_amd import binding as B
    rng = np.random.default_rng(9)
    for nb in (16, 4096, 17408, 69632):
        say(f"[pages] copy {nb}")
        pool = torch.randint(0, 256, (3, 40, nb), dtype=torch.uint8, device=dev)
        ids = rng.permutation(40)
        pairs = torch.tensor(ids[:30].reshape(15, 2).tolist() + [[-1, 3], [0, 40]], dtype=torch.int32, device=dev)
        for n in (0, 1, 15, 17, 99):           # counts past the list are cut; bad ids skipped
            want = pool.clone()
            for s, d in pairs[:min(n, 15)].tolist():
                want[:, d] = pool[:, s]
            got = pool.clone()
            B.dspark_cache_copy(got, pairs, torch.tensor([n], dtype=torch.int32, device=dev))
            assert torch.equal(got, want)
    one = torch.randint(0, 256, (40, 1024), dtype=torch.uint8, device=dev)
    got = one.clone()
    B.dspark_cache_copy(got, pairs, torch.tensor([15], dtype=torch.int32, device=dev))
    assert torch.equal(got[pairs[:15, 1].long()], one[pairs[:15, 0].long()])


def test_captured_round(dev):
    """fork, reserve, copy, commit and compact in one graph, replayed with
    eager work between: every replay equals the eager calls."""
    from semi_ar_draft_round_amd.cache import PagedCache
    rng = np.random.default_rng(11)
    R, gamma = 12, 16

    def make():
        c = PagedCache(2, R, 300, 160, 2, 64, page=16)
        c.pool.copy_(start)
        return c
    start = torch.randint(0, 256, (2, 160, 2 * 16 * 64 * 4), dtype=torch.uint8, device=dev)
    eager, graphed = make(), make()
    ell, acc, parent = (torch.zeros(R, dtype=torch.int32, device=dev) for _ in range(3))

    def step(c):
        c.fork(parent)
        c.reserve(ell, gamma)
        c.commit(acc)
        c.compact()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step(graphed)                                  # warm up on a copy that is reset below
        torch.cuda.synchronize()
        graphed.reset()
        graphed.pool.copy_(start)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(graphed)
    for i in range(6):
        say(f"[pages] replay {i}")
        ell.copy_(torch.tensor(rng.integers(-1, gamma + 1, R), dtype=torch.int32))
        acc.copy_(torch.tensor(rng.integers(0, gamma + 1, R), dtype=torch.int32))
        par = np.arange(R)
        par[rng.integers(0, R)] = rng.integers(-1, R)
        parent.copy_(torch.tensor(par, dtype=torch.int32))
        g.replay()
        step(eager)
        torch.cuda.synchronize()
        for a, b in ((eager.table, graphed.table), (eager.length, graphed.length), (eager.ref, graphed.ref),
                     (eager.bits, graphed.bits), (eager.pool, graphed.pool), (eager.ell, graphed.ell)):
            assert torch.equal(a, b)


def test_cache_object_refuses():
    from semi_ar_draft_round_amd.cache import PagedCache
    for bad in (dict(dim=100), dict(page=24), dict(n_pages=0), dict(layers=0), dict(window=-1), dict(fmt=3)):
        with pytest.raises(ValueError):
            PagedCache(**(dict(layers=1, slots=2, max_tokens=10, n_pages=4, heads_kv=1, dim=64) | bad))
