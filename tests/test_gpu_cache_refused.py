"""Whole rounds in which requests find no pages: they keep their cache and
their anchor, and go on from it once there are pages."""

import sys

import pytest

from semi_ar_draft_round_amd import workloads as W

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


@pytest.mark.parametrize("captured", [False, True])
def test_refused_in_a_round(captured, dev):
    """Four requests and pages for three; a target whose V is the token's row
    of a table, so that the cache says which token was run."""
    from semi_ar_draft_round_amd import binding as B
    from semi_ar_draft_round_amd import device_round as DR
    from semi_ar_draft_round_amd.cache import PagedCache
    say(f"[refused] captured {captured}")
    w = W.custom("refused_r4_g5_v300", R=4, gamma=5, V=300, r=32, d=64, dtype="f32", seed=81)
    d = DR.to_device(W.make_inputs(w), dev)
    Hq, D = 2, 64
    emb = torch.randn((w.V, Hq + 2, D), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(dev)
    head = torch.randn((Hq * D, w.V), generator=torch.Generator().manual_seed(7)).to(dev)
    c = PagedCache(1, w.R, 64, 3, 1, D, page=16)

    def forward(d, cache, ell):
        x = emb[torch.cat([d.x0.view(-1, 1), d.x], dim=1).view(-1).long()]
        q = cache.append(0, x[:, :Hq], x[:, Hq:Hq + 1], x[:, Hq + 1:])
        o = torch.zeros_like(q)
        cache.attend(0, q, out=o)
        d.target.copy_((o.view(q.shape[0], -1).float() @ head).view(d.target.shape))

    def step():
        DR.run_round_cached(d, c, forward)
        d.x0.copy_(d.next_tok)

    start = d.x0.clone()
    if captured:
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        c.reset()
        d.x0.copy_(start)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        step = g.replay
    for _ in range(2):                                  # the second round refuses it again
        step()
        torch.cuda.synchronize()
        ell, acc, length = c.ell.tolist(), d.n_acc.tolist(), c.length.tolist()
        say(f"  granted {ell} accepted {acc} length {length}")
        assert ell[3] == -1 and min(ell[:3]) >= 0 and int(c.status) == B.ENOPAGES
        assert acc[3] == -1 and min(acc[:3]) >= 0
        assert int(d.x0[3]) == int(start[3]) and length[3] == 0
    # it moves to slot 0, whose request is done: the round goes on from its anchor
    c.fork(torch.tensor([3, 1, 2, -1], dtype=torch.int32, device=dev))
    d.x0[0] = d.x0[3]
    step()
    torch.cuda.synchronize()
    assert int(c.ell[0]) >= 0 and int(c.length[0]) == int(d.n_acc[0]) + 1
    _, v = c.read(0, 1)
    assert torch.equal(v[0, 0, 0], emb[int(start[3]), Hq + 1])
