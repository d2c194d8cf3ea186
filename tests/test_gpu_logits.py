"""dspark_logits, _prompt and _commit against the float64 oracle.

Bound: each step of a logit's way is one fp32 rounding (2^-24) of what is there
by then: the quotient or product with the repetition, frequency * n + presence,
its difference, the sum of the biases (one rounding each) and the sum with it;
the largest magnitude on that way bounds them all.  bf16 rounds once more (2^-8
of the value)."""

import sys

import numpy as np
import pytest

from oracle import logits as OL
from semi_ar_draft_round_amd.workloads import bf16_bits, bf16_to_f32

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
    def __init__(self, dev, dt, R, gamma, V, ells, packed=True, nb=3, masked=True, drafts=True, history=True, seed=1):
        rng = np.random.default_rng(seed)
        self.__dict__.update(dev=dev, dt=dt, R=R, gamma=gamma, V=V, ells=ells, drafts=drafts, rng=rng)
        self.n = [min(max(e, -1), gamma) + 1 for e in ells]
        self.first = (np.cumsum([0] + self.n)[:-1] + 1).tolist() if packed else [r * (gamma + 1) for r in range(R)]
        self.rows = sum(self.n) + 2 if packed else R * (gamma + 1)
        x = (rng.standard_normal((self.rows, V)) * 3).astype(np.float32)
        self.nx = bf16_to_f32(bf16_bits(x)) if dt == "bf16" else x
        self.x = torch.from_numpy(self.nx).to(dev).to(torch.bfloat16 if dt == "bf16" else torch.float32)
        i32 = self.i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(dev)
        f32 = lambda a: torch.from_numpy(np.asarray(a, np.float32)).to(dev)
        tok = lambda *s: (V * rng.random(s) ** 3).astype(np.int32)
        self.nx0, self.nd = tok(R), tok(R, gamma)
        self.nx0[rng.random(R) < 0.2] = -1
        self.nd[rng.random((R, gamma)) < 0.1] = V
        if gamma > 3:
            self.nd[:, 2] = self.nd[:, 0]               # a draft that repeats
            self.nd[0, 1] = self.nx0[0]
        self.h = [OL.History(V) for _ in range(R)] if history else None
        if history:
            for h in self.h:
                h.start(tok(int(rng.integers(0, 40))))
                h.add(tok(int(rng.integers(0, 60))))
            self.h[0].count[: 5] = 32767
            self.state = torch.from_numpy(np.stack([h.words() for h in self.h]).view(np.int16)).to(dev)
        else:
            self.state = None
        self.rep, self.pres, self.freq = rng.uniform(0.7, 2, R), rng.uniform(-1, 2, R), rng.uniform(-0.5, 0.5, R)
        self.rep, self.pres, self.freq = (a.astype(np.float32) for a in (self.rep, self.pres, self.freq))
        self.t = [f32(a) for a in (self.rep, self.pres, self.freq)]
        self.nb = nb
        self.btok, self.b = tok(R, nb), (rng.standard_normal((R, nb)) * 5).astype(np.float32)
        if nb > 2:
            self.btok[:, 1] = self.btok[:, 0]           # a token with two biases
            self.btok[rng.random((R, nb)) < 0.1] = -1
            self.btok[0, 2] = V
        self.allowed = rng.random((self.rows, V)) < rng.choice([0.02, 0.5, 1.0], (self.rows, 1)) if masked else None
        if masked:
            W = -(-V // 32)
            bits = np.zeros((self.rows, W * 32), bool)
            bits[:, :V] = self.allowed
            bits[:, V:] = rng.random((self.rows, W * 32 - V)) < 0.5     # bits of no token
            self.mask = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32)).to(dev)
        else:
            self.mask = None
        self.kw = dict(row0=i32(self.first) if packed else None, repetition=self.t[0], presence=self.t[1],
                       frequency=self.t[2], bias_tok=i32(self.btok) if nb else None, bias=f32(self.b) if nb else None,
                       mask=self.mask)

    def call(self, logits, out):
        from semi_ar_draft_round_amd import binding as B
        return B.dspark_logits(logits, self.state, self.i32(self.ells), self.gamma, self.i32(self.nx0),
                               self.i32(self.nd) if self.drafts and self.gamma else None, out=out, **self.kw)

    def want(self):
        """Values and bounds [rows][V], NaN where a row is nobody's."""
        y, tol = np.full((self.rows, self.V), np.nan), np.zeros((self.rows, self.V))
        for r in range(self.R):
            biases = [(int(t), float(b)) for t, b in zip(self.btok[r], self.b[r])] if self.nb else []
            size = np.zeros(self.V)
            for t, b in biases:
                if 0 <= t < self.V:
                    size[t] += abs(b)
            for i in range(self.n[r]):
                k = self.first[r] + i
                follows = [int(self.nx0[r])] + ([int(t) for t in self.nd[r, :i]] if self.drafts else [])
                p = (float(self.rep[r]), float(self.pres[r]), float(self.freq[r]))
                h = self.h[r] if self.h else None
                y[k] = OL.row(self.nx[k], h, follows, *p, biases, self.allowed[k] if self.allowed is not None else None)
                plain = OL.row(np.abs(self.nx[k]), None, follows, *p, [], None) * max(p[0], 1 / p[0])
                if h is not None:
                    plain = plain + (h.count + len(follows)) * abs(p[2]) + abs(p[1])
                tol[k] = (6 + self.nb) * 2.0 ** -24 * (plain + size) + 1e-37
        if self.dt == "bf16":
            tol = tol * 2 + np.abs(np.where(np.isfinite(y), y, 0)) * 2.0 ** -8
        return y, tol

    def check(self):
        y, tol = self.want()
        live = ~np.isnan(y).all(axis=1)
        fill = torch.full_like(self.x, 7.0)
        for inplace in (False, True):
            src = self.x.clone()
            out = src if inplace else fill.clone()
            self.call(src, out)
            torch.cuda.synchronize()
            got = out.float().cpu().numpy().astype(np.float64)
            assert np.array_equal(got[~live], (self.nx if inplace else fill.float().cpu().numpy())[~live])
            g, w = got[live], y[live]
            assert np.array_equal(np.isneginf(g), np.isneginf(w))
            fine = np.isfinite(w)
            err = np.abs(np.where(fine, g, 0) - np.where(fine, w, 0))
            assert np.all(err <= tol[live]), float((err / tol[live]).max())
            if not inplace:
                assert torch.equal(src, self.x)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R,gamma,V,ells,packed", [(1, 0, 2, [0], False), (1, 4, 7, [4], True), (3, 4, 1024, [4, -1, 2], True),
                                                   (2, 16, 2047, [16, 9], False), (5, 2, 2049, [0, 5, -3, 2, 1], False),
                                                   (2, 3, 5003, [3, 3], True), (4, 1, 33000, [1, 0, -1, 1], True),
                                                   (1, 200, 301, [200], True), (1, 1023, 40, [1023], False),
                                                   (300, 2, 50, [r % 4 - 1 for r in range(300)], True)])
def test_logits_against_oracle(R, gamma, V, ells, packed, dt, dev):
    say(f"[logits] {dt} {R} {gamma} {V}")
    Case(dev, dt, R, gamma, V, ells, packed, seed=V).check()


@pytest.mark.parametrize("kw", [dict(nb=0), dict(masked=False), dict(drafts=False), dict(history=False),
                                dict(nb=0, masked=False, history=False), dict(nb=200), dict(nb=65)])
def test_parts_alone(kw, dev):
    say(f"[logits] {kw}")
    for dt in ("f32", "bf16"):
        Case(dev, dt, 3, 5, 999, [5, 2, 0], seed=9, **kw).check()


def test_without_any_condition_a_row_is_itself(dev):
    say("[logits] identity")
    c = Case(dev, "bf16", 2, 3, 1001, [3, 1], nb=0, masked=False)
    c.kw.update(repetition=None, presence=None, frequency=None)
    out = c.call(c.x, torch.full_like(c.x, 7.0))
    for f, n in zip(c.first, c.n):
        assert torch.equal(out[f:f + n], c.x[f:f + n])


def test_not_finite_logits_and_rows_that_allow_nothing(dev):
    say("[logits] not finite")
    c = Case(dev, "f32", 1, 2, 600, [2], nb=0, packed=False, seed=3)
    c.x[0, :100], c.x[0, 100:200], c.x[1, :300] = float("inf"), float("nan"), -float("inf")
    c.mask[2] = 0
    c.mask[:2] = -1
    c.nx[:] = c.x.cpu().numpy()
    out = c.call(c.x, torch.empty_like(c.x)).cpu().numpy()
    assert np.all(out[0, :100] == np.inf) and np.all(np.isnan(out[0, 100:200])) and np.all(out[1, :300] == -np.inf)
    assert np.isfinite(out[0, 200:]).all() and np.isfinite(out[1, 300:]).all() and np.all(out[2] == -np.inf)
    c.mask[:] = 0
    assert np.all(c.call(c.x, torch.empty_like(c.x)).cpu().numpy() == -np.inf)   # NaN and inf too


@pytest.mark.parametrize("V", [2, 31, 1000, 8191, 8192, 8193, 16384, 16385, 40007])
def test_history(V, dev):
    """Prompts of every length, slots left alone, rounds with repeated tokens."""
    from semi_ar_draft_round_amd.logits import Conditions
    say(f"[logits] history {V}")
    rng = np.random.default_rng(V)
    R, gamma = 6, 80
    c = Conditions(R, V, device=dev)
    h = [OL.History(V) for _ in range(R)]
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(dev)
    tok = lambda n: rng.integers(-2, V + 2, n).astype(np.int32) if n % 2 else (V * rng.random(n) ** 4).astype(np.int32)
    for turn in range(3):
        counts = [0, 5, 1000, -1, 33, int(rng.integers(0, 500))]
        tokens = tok(sum(max(n, 0) for n in counts) + 7)
        start = (np.cumsum([3] + [max(n, 0) for n in counts])[:-1]).astype(int)
        c.prompt(i32(tokens), i32(start), i32(counts))
        for r, n in enumerate(counts):
            if n >= 0:
                h[r].start(tokens[start[r]:start[r] + n].tolist())
        for _ in range(3):
            x0, x = tok(R), tok(R * gamma).reshape(R, gamma)
            x[2] = x[2, 0]                                   # one token all over
            ell, acc = [80, 0, 80, -1, 70, 5], [80, 3, 79, 4, 64, -1]
            c.commit(i32(ell), i32(acc), i32(x0), i32(x))
            for r in range(R):
                if ell[r] >= 0:
                    h[r].add([int(x0[r])] + x[r, :min(max(acc[r], 0), ell[r])].tolist())
            torch.cuda.synchronize()
            got = c.state.cpu().numpy().view(np.uint16)
            assert np.array_equal(got, np.stack([a.words() for a in h]))
    # past the list's ends, and none at all
    c.prompt(i32([1, 1]), i32([-1, 1, 2, 5, 0, 2 ** 31 - 1]), i32([2, 100, 3, 1, 0, 2 ** 31 - 1]))
    for a, t in zip(h, ([1], [1], [], [], [], [])):
        a.start(t)
    assert np.array_equal(c.state.cpu().numpy().view(np.uint16), np.stack([a.words() for a in h]))
    c.prompt(torch.empty(0, dtype=torch.int32, device=dev), i32([0] * R), i32([0] + [-1] * 5))
    c.commit(i32([0] * R), i32([0] * R), i32([1] * R))       # no drafts
    h[0].start([])
    for a in h:
        a.add([1])
    assert np.array_equal(c.state.cpu().numpy().view(np.uint16), np.stack([a.words() for a in h]))


def test_counts_stop(dev):
    from semi_ar_draft_round_amd import binding as B
    say("[logits] counts stop")
    state = torch.tensor([[32766, -2, 0, 32767]], dtype=torch.int16, device=dev)   # -2: in the prompt, 32766
    one = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
    B.dspark_logits_commit(state, one(5), one(5), one(0), torch.tensor([[0, 1, 1, 3, 2]], dtype=torch.int32, device=dev))
    assert state.tolist() == [[32767, -1, 1, 32767]]


def test_fork_of_conditions(dev):
    from semi_ar_draft_round_amd.logits import Conditions
    say("[logits] fork")
    c = Conditions(4, 50, biases=2, device=dev)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
    c.prompt(i32(3, 4, 5, 6), i32(0, 1, 2, 3), i32(1, 1, 1, 1))
    c.repetition.copy_(torch.tensor([1.1, 1.2, 1.3, 1.4], device=dev))
    before = c.state.clone()
    c.fork(i32(1, 0, -1, 9))
    assert torch.equal(c.state[:2], before[[1, 0]]) and not c.state[2].any() and torch.equal(c.state[3], before[3])
    assert torch.allclose(c.repetition.cpu(), torch.tensor([1.2, 1.1, 1.3, 1.4]))


def test_captured_and_replayed(dev):
    from semi_ar_draft_round_amd.logits import Conditions
    say("[logits] captured")
    rng = np.random.default_rng(4)
    R, gamma, V = 3, 4, 5000
    c = Conditions(R, V, biases=2, device=dev)
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(dev)
    tokens, start, count = i32(rng.integers(0, V, 60)), i32([0, 20, 40]), i32([20, 20, 20])
    ell, acc, x0, x = i32([4, 2, -1]), i32([3, 2, 0]), i32(rng.integers(0, V, R)), i32(rng.integers(0, V, (R, gamma)))
    c.presence.fill_(0.5)
    logits = torch.randn((R, gamma + 1, V), device=dev).to(torch.bfloat16)
    out = logits.clone()

    def step():
        c.prompt(tokens, start, count)
        c.apply(logits, ell, gamma, x0, x, out=out)
        c.commit(ell, acc, x0, x)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    want, state = out.clone(), c.state.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(4):
        out.copy_(logits)
        c.state.fill_(77)
        g.replay()
        torch.randn(1000, device=dev).sum()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(c.state, state)


def test_rows_past_32_bit_offsets(dev):
    """More than 2^32 bytes of logits: the last rows are as they are alone."""
    from semi_ar_draft_round_amd import binding as B
    say("[logits] far rows")
    V, rows = 151936, 15000
    big = torch.empty((rows, V), dtype=torch.bfloat16, device=dev)
    c = Case(dev, "bf16", 2, 3, V, [3, 2], seed=5)
    at = rows - c.rows
    big[at:] = c.x
    c.kw["mask"] = None
    alone = c.call(c.x, torch.full_like(c.x, 7.0))
    c.kw["row0"] = c.kw["row0"] + at
    c.call(big, big)
    for f, n in zip(c.first, c.n):
        assert torch.equal(big[at + f:at + f + n], alone[f:f + n])
