"""The masses that PagedCache keeps with a budget: each is what its page's tokens
got, through commits, evictions and forks."""

import sys

import pytest

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


D, HQ, GAMMA, P = 64, 4, 20, 16


class Rows:
    """Rows by request and position, whatever round brings them."""

    def __init__(self, dev, slots, seed):
        g = torch.Generator().manual_seed(seed)
        self.x = torch.randn((slots, 200, HQ + 2, D), generator=g).to(torch.bfloat16).to(dev)
        self.dev = dev

    def round(self, c, ell, n_acc, spoil=None):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=self.dev)
        length = c.length.tolist()
        c.reserve(i32(ell), GAMMA)
        assert c.ell.tolist() == ell
        x = torch.stack([self.x[r, n:n + GAMMA + 1] for r, n in enumerate(length)]).view(-1, HQ + 2, D).clone()
        if spoil is not None:
            x[spoil] = float("nan")
        for layer in range(c.pool.shape[0]):
            c.attend(layer, c.append(layer, x[:, :HQ], x[:, HQ:HQ + 1], x[:, HQ + 1:]))
        before = c.mass.clone()
        c.commit(i32(n_acc))
        torch.cuda.synchronize()
        return before


@pytest.mark.parametrize("fade,window", [(1.0, 0), (0.75, 0), (1.0, 20)])
def test_a_rejected_page_leaves_no_mass(fade, window, dev):
    """Pages of rejected drafts go with the commit, and their mass with them: what
    is written there later starts from nothing."""
    from semi_ar_draft_round_amd.cache import PagedCache
    say(f"[mass] rejected {fade} {window}")
    c, rows = PagedCache(2, 2, 150, 30, 1, D, page=P, budget=50, fade=fade, window=window), Rows(dev, 2, 1)
    for _ in range(2):
        rows.round(c, [14, 20], [14, 20])
    before = rows.round(c, [20, 20], [1, 0])         # tokens 30 .. 50 and 42 .. 62: 32 and 43 stay
    assert c.length.tolist() == [32, 43]
    assert (before[0, 2:4] > 0).all() and before[1, 3] > 0
    assert not c.mass[0, 2:].any() and not c.mass[1, 3:].any()
    if window:
        assert (c.table[1, 0] < 0) and c.mass[1, 0] == 0
    # the next round's pages start from nothing: no more than the rows' shares
    m = c.mass.clone()
    rows.round(c, [0, 10], [0, 10])
    assert c.length.tolist() == [33, 54]
    gained = (c.mass - m * fade).sum(dim=1)
    want = torch.tensor([1.0, 11.0], device=dev) * HQ * 2
    got = gained if not window else gained[:1]
    # every row and head shares out one a layer; a window's release takes its page's share along
    assert bool(((got - want[:len(got)]).abs() < 1e-3 * want[:len(got)]).all()), gained
    assert 0 < float(c.mass[0, 2]) <= HQ * 2 * 1.001


def test_a_rejected_row_that_is_not_finite(dev):
    """A NaN among rejected rows: the mass of the pages that it alone wrote is 0
    again, that of those it saw is NaN until it is weighed with keep = 0."""
    from semi_ar_draft_round_amd.cache import PagedCache
    say("[mass] NaN")
    for fmt in (1, 4):
        c, rows = PagedCache(1, 1, 150, 10, 1, D, page=P, fmt=fmt, budget=50, fade=0.0), Rows(dev, 1, 2)
        rows.round(c, [19], [19])
        before = rows.round(c, [20], [3], spoil=20)
        assert torch.isnan(before[0, :3]).all()
        assert torch.isnan(c.mass[0, :2]).all() and not c.mass[0, 2:].any()
        rows.round(c, [2], [2])
        assert torch.isfinite(c.mass).all() and abs(float(c.mass.sum()) - 3 * HQ) < 1e-3 * 3 * HQ


@pytest.mark.parametrize("page", [16, 64])
def test_keep_0_takes_any_mass_for_0(page, dev):
    """Entries that rows see, that lie between the first tokens and the window,
    and behind the last row: NaN and infinities there before make no difference,
    and requests without rows are left alone."""
    from test_gpu_cache_weigh import Case
    say(f"[mass] keep 0, pages of {page}")
    c = Case(dev, 1, [700, 40, 90], [16, -1, 3], 4, 2, 64, page, 16, window=100, sinks=20, more=300, seed=3)
    zero = torch.zeros(c.old.shape, device=dev)
    want = c.call(0.0, zero.clone())
    assert (want[0, 2:500 // page] == 0).all() and (want[0] > 0).any() and (want[:, -1] == 0).all()
    for x in (float("nan"), float("inf"), -float("inf")):
        got = c.call(0.0, torch.full_like(zero, x))
        assert (got[[0, 2]] == want[[0, 2]]).all()
        assert (got[1] == x).all() or (x != x and (got[1] != got[1]).all())


def test_a_fork_takes_the_budget_along(dev):
    """Requests of different budgets change places: each is held to its own at
    the next commit, as if it had stayed where it was."""
    from semi_ar_draft_round_amd.cache import PagedCache
    say("[mass] budgets")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
    for swap in (False, True):
        c, rows = PagedCache(1, 4, 150, 60, 1, D, page=P, budget=2 ** 31 - 1), Rows(dev, 4, 3)
        c.budget.copy_(i32(2, 50, -1, 3))
        for _ in range(4):
            rows.round(c, [20] * 4, [20] * 4)
        assert [int((t >= 0).sum()) for t in c.table] == [2, 6, 6, 3]
        if swap:
            c.fork(i32(1, 0, 2, -1))
            rows.x[[0, 1]] = rows.x[[1, 0]]
            assert c.budget.tolist() == [50, 2, -1, 3]
        rows.round(c, [20] * 4, [20] * 4)
        held = [int((t >= 0).sum()) for t in c.table]
        assert held == ([7, 2, 7, 2] if swap else [2, 7, 7, 3])
