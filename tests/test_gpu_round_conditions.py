"""Whole rounds over a cache with a budget of pages and requests with
conditions: drafted, verified against the conditioned logits, committed and
evicted, eagerly and from a captured graph."""

import sys

import numpy as np
import pytest

from oracle import logits as OL
from semi_ar_draft_round_amd import workloads as W

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

R, GAMMA, V, HQ, D, P, BUDGET, LAYERS = 5, 6, 401, 4, 64, 16, 3, 2


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from semi_ar_draft_round_amd import binding
    binding.load_library()
    return torch.device("cuda:0")


class Server:
    """A small target whose projections are tables by token; a grammar that
    allows after n tokens only those with v % 3 == n % 3; a presence penalty
    that no logit outweighs, so that no token comes twice."""

    def __init__(self, dev, dtype, fmt):
        from semi_ar_draft_round_amd import device_round as DR
        from semi_ar_draft_round_amd.cache import PagedCache
        from semi_ar_draft_round_amd.logits import Conditions
        w = W.custom("conditions", R=R, gamma=GAMMA, V=V, r=32, d=64, dtype=dtype, seed=91)
        self.d = DR.to_device(W.make_inputs(w), dev)
        g = torch.Generator().manual_seed(6)
        self.emb = [torch.randn((V, HQ + 2, D), generator=g).to(torch.bfloat16).to(dev) for _ in range(LAYERS)]
        self.head = (torch.randn((HQ * D, V), generator=g) * 0.3).to(dev)
        self.cache = PagedCache(LAYERS, R, 300, R * 19, 1, D, page=P, fmt=fmt, budget=BUDGET, fade=0.9, keep_first=4,
                                keep_last=20)
        self.cond = Conditions(R, V, biases=1, device=dev)
        self.cond.presence.fill_(1e4)
        self.cond.bias_tok.fill_(7)
        self.cond.bias.fill_(2.0)
        allowed = np.zeros((3, -(-V // 32) * 32), bool)
        for a in range(3):
            allowed[a, a:V:3] = True
        self.grammar = torch.from_numpy(np.packbits(allowed, axis=1, bitorder="little").view(np.int32)).to(dev)
        self.mask = torch.zeros((R * (GAMMA + 1), self.grammar.shape[1]), dtype=torch.int32, device=dev)
        self.at = torch.arange(GAMMA + 1, device=dev)
        self.d.x0.copy_(torch.arange(R, device=dev) * 3 + 2)      # token 0 of a request: v % 3 == 2, as after -1
        self.d.x.zero_()

    def forward(self, d, cache, ell):
        # row i of a request follows len + 1 + i tokens
        n = (cache.length.view(-1, 1) + self.at).view(-1) % 3
        self.mask.copy_(self.grammar[n.long()])
        tok = torch.cat([d.x0.view(-1, 1), d.x], dim=1).view(-1).long().clamp(0, V - 1)
        out = 0
        for layer in range(LAYERS):
            x = self.emb[layer][tok]
            q = cache.append(layer, x[:, :HQ], x[:, HQ:HQ + 1], x[:, HQ + 1:])
            o = torch.zeros_like(q)
            cache.attend(layer, q, out=o)
            out = out + o.float()
        d.target.copy_((out.view(out.shape[0], -1) @ self.head).view(d.target.shape))

    def step(self):
        from semi_ar_draft_round_amd import device_round as DR
        DR.run_round_cached(self.d, self.cache, self.forward, conditions=self.cond, mask=self.mask)
        self.d.x0.copy_(self.d.next_tok)

    def tensors(self):
        c = self.cache
        return c.table, c.length, c.ref, c.bits, c.mass, c.freed, self.cond.state, self.d.x, self.d.x0, self.d.n_acc


@pytest.mark.parametrize("dtype,fmt", [("f32", 4), ("bf16", 1), ("bf16", 4), ("f32", 2)])
def test_rounds(dtype, fmt, dev):
    say(f"[round] {dtype} {fmt}")
    s = Server(dev, dtype, fmt)
    start = [t.clone() for t in s.tensors()]
    history = [OL.History(V) for _ in range(R)]
    answer = [[int(t)] for t in s.d.x0]
    states, freed = [], 0
    for _ in range(110):
        before = s.d.x0.tolist()
        s.step()
        torch.cuda.synchronize()
        x, acc, ell = s.d.x.tolist(), s.d.n_acc.tolist(), s.cache.ell.tolist()
        for r in range(R):
            assert 0 <= acc[r] <= ell[r]
            new = x[r][:acc[r]] + [int(s.d.x0[r])]
            history[r].add([before[r]] + x[r][:acc[r]])
            for t in new:
                assert t % 3 == (len(answer[r]) - 1) % 3, "the grammar"
                assert t not in answer[r], "the penalty"
                answer[r].append(t)
            assert int(s.cache.length[r]) == len(answer[r]) - 1
        got = s.cond.state.cpu().numpy().view(np.uint16)
        assert np.array_equal(got, np.stack([h.words() for h in history]))
        table, ref, length = s.cache.table.cpu().numpy(), s.cache.ref.cpu().numpy(), s.cache.length.tolist()
        count = np.zeros(len(ref), int)
        np.add.at(count, table[table >= 0], 1)
        assert np.array_equal(count, ref)
        for r, n in enumerate(length):
            held = np.flatnonzero(table[r] >= 0)
            used = -(-n // P)
            fixed = sum(not (i * P >= 4 and (i + 1) * P <= n - 20) for i in range(used))
            assert len(held) <= max(BUDGET, fixed) and (used == 0 or held[-1] == used - 1)
            assert not used or n <= 20 or held[0] == 0               # the first tokens stay
        freed += int(s.cache.freed.sum())
        states.append([t.clone() for t in s.tensors()])
    assert freed > R and min(length) > (BUDGET + 1) * P
    say(f"  lengths {length}, pages freed {freed}")

    # the same rounds from a graph
    def rewind():
        for t, x in zip(s.tensors(), start):
            t.copy_(x)
    rewind()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        s.step()
    rewind()
    for want in states:
        g.replay()
        torch.randn(1000, device=dev).sum()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(s.tensors(), want))


def test_fork_takes_weights_along(dev):
    from semi_ar_draft_round_amd.cache import PagedCache
    say("[round] fork")
    c = PagedCache(1, 3, 100, 20, 1, 64, page=16, fmt=4, budget=2)
    c.mass.copy_(torch.arange(21, device=dev).view(3, 7))
    c.fork(torch.tensor([2, -1, 7], dtype=torch.int32, device=dev))
    assert c.mass.tolist() == [[float(x) for x in range(14, 21)], [0.0] * 7, [float(x) for x in range(14, 21)]]
    c.reset()
    assert not c.mass.any()


def test_a_budget_leaves_the_windows_first_tokens(dev):
    """What the attention's window keeps visible is not evicted, whether or not
    it got any weight."""
    from semi_ar_draft_round_amd.cache import PagedCache
    say("[round] budget and window")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    c = PagedCache(1, 2, 300, 40, 1, 64, page=16, window=64, sinks=20, budget=3)
    x = torch.ones((2 * 100, 1, 64), dtype=torch.bfloat16, device=dev)
    c.reserve(i32([99, 99]), 99)
    c.attend(0, c.append(0, x, x, x))
    c.mass.copy_(torch.arange(c.mass.shape[1], device=dev).expand(2, -1))
    c.commit(i32([99, 70]))
    torch.cuda.synchronize()
    assert (c.table[:, :2] >= 0).all()
    assert [(row >= 0).sum().item() for row in c.table] == [3, 3]
