"""Long caches, so that work groups take long runs, against float64 on the
device over the values that dspark_cache_read gives: dspark_cache_weigh over
pages of all formats, and dspark_cache_attention over 8-bit pages, whose tiles
of 256-dim heads come through a ring in LDS.

Bounds: of a weight as in test_gpu_cache_weigh, of attention as in
test_gpu_cache_attention; the sum of magnitudes of a score is at most the
product of the norms."""

import numpy as np
import pytest

import test_gpu_cache_attention as A
from cache8_cases import FP8
from cache_cases import BF16, F32, FP4
from test_gpu_cache8 import Case8, i32
from test_gpu_cache_attention import say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from semi_ar_draft_round_amd import binding
    binding.load_library()
    return torch.device("cuda:0")


def filled(dev, fmt, total, Hkv, D, P, seed, more=0):
    """A pool with `total[r]` tokens of every request, their table."""
    from semi_ar_draft_round_amd import binding as B
    R, T = len(total), max(total)
    g = torch.Generator(device=dev).manual_seed(seed)
    mp = -(-T // P) + more
    pool = torch.full((R * mp, B.dspark_cache_page_bytes(fmt, Hkv, D, P)), 0xFF, dtype=torch.uint8, device=dev)
    table = torch.randperm(R * mp, generator=g, device=dev).to(torch.int32).view(R, mp)
    C = min(1024, T)
    for at in range(0, T, C):
        x = torch.randn((R * C, 1 + 2 * Hkv, D), generator=g, device=dev).to(torch.bfloat16)
        B.dspark_cache_append(x[:, :1], x[:, 1:1 + Hkv], x[:, 1 + Hkv:], pool, table, i32([min(at, t) for t in total], dev),
                              i32([min(t - at, C) - 1 if t > at else -1 for t in total], dev), C - 1, fmt=fmt, page=P)
    return pool, table, g


WEIGH = {  # lens, ells, Hq, Hkv, D, P, window, sinks, the share of pages that are gone
    "ragged": ([20_011, 19_000, 300, 12_345] * 4, [16, 0, 16, 5] * 4, 8, 2, 128, 64, 0, 0, 0.0),
    "one-head": ([600_000], [0], 1, 1, 64, 16, 0, 0, 0.1),                  # more than 64 chunks a work group, twice over
    "two-rows-a-head": ([270_001], [1], 2, 1, 64, 16, 0, 0, 0.0),
    "three-heads": ([90_000, 7], [3, 3], 6, 3, 128, 16, 0, 0, 0.5),
    "d256": ([9_000, 6_000, 12_000, 100] * 2, [16, 3, 0, -1] * 2, 8, 2, 256, 32, 0, 0, 0.0),
    "d256-one-head": ([250_000], [4], 1, 1, 256, 64, 0, 0, 0.9),
    "window": ([20_000, 15_000, 9_100, 4_000] * 2, [16, 0, 9, 3] * 2, 8, 2, 64, 16, 9_000, 300, 0.0),
    "window-large-pages": ([40_000] * 6, [7] * 6, 4, 4, 128, 128, 20_000, 1_000, 0.2),
    "many-requests": ([(r * 37) % 500 for r in range(700)], [r % 4 - 1 for r in range(700)], 4, 2, 64, 32, 0, 0, 0.0),
    "rows-in-blocks": ([3_000, 2_500], [400, 0], 8, 1, 128, 64, 0, 0, 0.0),  # more row blocks than waves
}


@pytest.mark.parametrize("fmt", [BF16, FP4, FP8])
@pytest.mark.parametrize("name", WEIGH)
def test_weigh(name, fmt, dev):
    from semi_ar_draft_round_amd import binding as B
    lens, ells, Hq, Hkv, D, P, window, sinks, gone = WEIGH[name]
    say(f"[weigh] long {name} {fmt}")
    R, G, n = len(lens), Hq // Hkv, [e + 1 for e in ells]
    total = [a + b for a, b in zip(lens, n)]
    pool, table, g = filled(dev, fmt, total, Hkv, D, P, 17, more=3)
    reads = table.clone()
    there = torch.rand(table.shape, generator=g, device=dev) >= gone
    there[:, 0] = True
    for r in range(R):
        there[r, lens[r] // P:] = True                      # a row's own page
    table = torch.where(there, table, -2).to(torch.int32)
    first = np.cumsum([0] + n)[:-1].tolist()
    q = torch.randn((max(1, sum(n)), Hq, D), generator=g, device=dev).to(torch.bfloat16)
    old = torch.rand(table.shape, generator=g, device=dev) * 4
    scale, keep = D ** -0.5, 0.75
    lse = torch.full((q.shape[0], Hq), float("nan"), device=dev)
    want, bound = old.double().clone(), torch.zeros(old.shape, dtype=torch.float64, device=dev)
    for r in range(R):
        if n[r] == 0:
            continue
        N = total[r]
        k, _ = B.dspark_cache_read(pool, reads[r:r + 1].contiguous(), None, i32([N], dev), N, fmt=fmt, page=P,
                                   heads_kv=Hkv, dim=D)
        k = k[0].double().permute(1, 2, 0).contiguous()                          # [Hkv][D][N]
        mine = slice(first[r], first[r] + n[r])
        x = q[mine].double().view(n[r], Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, -1, D)
        s = (torch.bmm(x, k) * scale).view(Hkv, n[r], G, N)
        j, pos = torch.arange(N, device=dev), lens[r] + torch.arange(n[r], device=dev)[:, None]
        see = (j <= pos) & there[r, j // P]
        if window:
            see &= (j > pos - window) | (j < sinks)
        s.masked_fill_(~see[None, :, None], float("-inf"))
        z = torch.logsumexp(s, -1).float()                                       # what attention would give
        lse[mine] = z.permute(1, 0, 2).reshape(n[r], Hq)
        w = torch.exp(s - z.double()[..., None]).sum(dim=(0, 1, 2))
        pages = -(-N // P)
        w = torch.nn.functional.pad(w, (0, pages * P - N)).view(pages, P).sum(1)
        want[r] *= keep
        want[r, :pages] += w
        mag = float(x.norm(dim=-1).max() * k.norm(dim=1).max()) * scale
        rel = 2 * ((D + 8) * F32 * mag + 2.0 ** -23 * float(z.abs().max())) + 2.0 ** -22 + (n[r] * Hq * P + 64) * F32
        bound[r] = rel * want[r] + 1e-30
        del k, s
    args = dict(keep=keep, fmt=fmt, page=P, heads_kv=Hkv, window=window, sinks=sinks, row0=i32(first, dev))
    got = [B.dspark_cache_weigh(q, lse, pool, table, i32(lens, dev), i32(ells, dev), max(ells), old.clone(), **args)
           for _ in range(2)]
    torch.cuda.synchronize()
    assert torch.equal(*got)
    for r in range(R):
        if n[r] == 0:
            assert torch.equal(got[0][r], old[r])
    err = (got[0].double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound.clamp(min=1e-30)).max())
    say(f"  worst error {float((err / bound.clamp(min=1e-30)).max()):.3f} of its bound")


@pytest.mark.parametrize("case", A.LARGE, ids=["runs", "parts", "odd-parts", "row-tiles", "idle", "d256", "r4096"])
def test_attention_work_shared_out(case, dev):
    A.test_work_shared_out(case, FP8, dev)


# rows a head: 4 (the four waves along the tokens), 36 .. 64 (two), 100 .. 128 (one), and two blocks
@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("ells", [[0, 0, 0, 0, 0], [11, 8, 15, 11, 9], [24, 31, 29, 30, 31], [31, 40, 0, 9, -1]],
                         ids=["rows4", "rows64", "rows128", "blocks"])
def test_attention_through_the_ring(ells, P, dev):
    """8-bit heads of 256 dims, runs of more than 64 rounds of the ring."""
    A.test_work_shared_out(([60_000, 59_990, 50_001, 40_017, 47_999], ells, 32, 8, 256, P, max(ells)), FP8, dev)


@pytest.mark.parametrize("D", [128, 256])
def test_streams_graphs_and_repeats(D, dev):
    """Twice, with a dirty workspace, two calls at once with workspaces of their
    own, and captured with eager calls between the replays: the same bits."""
    from semi_ar_draft_round_amd import binding as B
    say(f"[attention] 8 bits, streams {D}")
    a = Case8(dev, [2000, 333, 40], [16, 16, 3], 8, 2, D, 64, 16, seed=20)
    b = Case8(dev, [1500, 700], [2, 16], 14, 2, D, 16, 16, 200, 4, seed=21)
    blank = lambda x: torch.zeros((x.rows, x.Hq), device=dev)
    want = [x.call(lse=blank(x)) for x in (a, b)]
    live = [[f + i for f, n in zip(x.first, x.n) for i in range(n)] for x in (a, b)]

    def same(i, got):
        assert torch.equal(want[i][0][live[i]], got[0][live[i]]) and torch.equal(want[i][1][live[i]], got[1][live[i]])

    for i, x in enumerate((a, b)):
        size = B.dspark_cache_workspace_size(B.CACHE_WS_ATTENTION, len(x.lens), x.gamma, x.Hq, x.Hkv, x.D)
        same(i, x.call(lse=blank(x), ws=torch.full((size,), 0xFF, dtype=torch.uint8, device=dev)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        torch.cuda.synchronize()
        for x, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                got.append(x.call(lse=blank(x)))
        torch.cuda.synchronize()
        same(0, got[0])
        same(1, got[1])
    outs = [(torch.zeros_like(w[0]), torch.zeros_like(w[1])) for w in want]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.call(*outs[0])
        b.call(*outs[1])
    for _ in range(4):
        for o in outs:
            o[0].zero_(), o[1].zero_()
        g.replay()
        same(0, a.call(lse=blank(a)))
        torch.cuda.synchronize()
        same(0, outs[0])
        same(1, outs[1])
