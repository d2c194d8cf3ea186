"""The cache's operators as a serving process uses them together: rounds of
reserve, append, attention and commit with forks and compactions between, and
the whole draft-and-verify round with a target that reads the cache.

Dense K and V per request are kept on the host.  The attention is compared
with the float64 oracle over the values that dspark_cache_read gives for the
cached tokens, within cache_cases.attention_tolerance; a 4-bit V reads back
rounded to bf16, which adds half a step, 2^-8 of sum_j p_j |v_j|."""

import sys

import numpy as np
import pytest

from cache_cases import BF16, F32, FP4, HALF, attention_tolerance, bf
from oracle import cache as OC
from semi_ar_draft_round_amd import workloads as W
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


def check_attention(o, q, k, v, pos, scale, window, sinks, fmt):
    want, _ = OC.attention(q, k, v, pos, scale, window, sinks)
    tol, _ = attention_tolerance(q, k, v, pos, scale, window, sinks, want)
    if fmt == FP4:
        tol = tol + HALF * OC.attention(q, k, np.abs(v), pos, scale, window, sinks)[0]
    err = np.abs(o - want)
    assert np.all(err <= tol), float((err / tol).max())


class Host:
    """Dense tokens of every request and layer beside a PagedCache."""

    def __init__(self, cache, slots, layers, Hkv, D):
        self.c, self.R, self.layers = cache, slots, layers
        self.kv = [[(np.zeros((0, Hkv, D)), np.zeros((0, Hkv, D))) for _ in range(layers)] for _ in range(slots)]

    def length(self, r):
        return len(self.kv[r][0][0])

    def take_rows(self, layer, ell, gamma):
        """Reads the rows append has just written; -> per request (k, v) of all tokens."""
        start = self.c.length
        k, v = self.c.read(layer, gamma + 1, start, (ell + 1).to(start.device))
        k, v = back(k), back(v)
        out = []
        for r, e in enumerate(ell.tolist()):
            a, b = self.kv[r][layer]
            out.append((np.concatenate([a, k[r, :e + 1]]), np.concatenate([b, v[r, :e + 1]])))
        return out, k, v

    def fork(self, parent):
        old = list(self.kv)
        for r, p in enumerate(parent):
            if p == -1:
                self.kv[r] = [(a[:0], b[:0]) for a, b in old[r]]
            elif 0 <= p < self.R:
                self.kv[r] = list(old[p])


@pytest.mark.parametrize("fmt,window,sinks", [(BF16, 0, 0), (BF16, 40, 5), (FP4, 0, 0), (FP4, 40, 5)])
def test_rounds_with_forks_and_compaction(fmt, window, sinks, dev):
    from semi_ar_draft_round_amd.cache import PagedCache
    say(f"[round] fmt {fmt} window {window}")
    rng = np.random.default_rng(40 + fmt + window)
    R, layers, Hq, Hkv, D, P, gamma = 6, 2, 6, 2, 128 if window else 64, 16, 21
    c = PagedCache(layers, R, 400, 70, Hkv, D, page=P, fmt=fmt, window=window, sinks=sinks)
    c.pool.fill_(0xFF)                                        # NaNs wherever nothing was written
    host = Host(c, R, layers, Hkv, D)
    freq = 1e4 ** (-2.0 * np.arange(D // 2) / D)
    tfreq = torch.from_numpy(freq).to(dev)
    scale = D ** -0.5
    for step in range(9):
        say(f"  step {step}, tokens {[host.length(r) for r in range(R)]}")
        ask = torch.tensor(rng.integers(-1, gamma + 1, R), dtype=torch.int32, device=dev)
        ell_t = c.reserve(ask, gamma)
        ell = ell_t.cpu()
        n = (ell + 1).numpy()
        first = np.cumsum(n) - n + 1                          # a row in front belongs to nobody
        rows = int(n.sum()) + 2
        row0 = torch.tensor(first, dtype=torch.int32, device=dev)
        wb, w = bf(1 + 0.3 * rng.standard_normal((2, D)))
        wq, wk = t16(wb[0], dev), t16(wb[1], dev)
        after = []
        for layer in range(layers):
            xb, x = bf(rng.standard_normal((rows, Hq + 2 * Hkv, D)))
            xt = t16(xb, dev)
            q = c.append(layer, xt[:, :Hq], xt[:, Hq:Hq + Hkv], xt[:, Hq + Hkv:], wq=wq, wk=wk, freq=tfreq, row0=row0)
            out = torch.full((rows, Hq, D), 5.0, dtype=torch.bfloat16, device=dev)
            c.attend(layer, q, row0=row0, out=out)
            dense, kr, vr = host.take_rows(layer, ell, gamma)
            o, qn = back(out), back(q)
            for r in range(R):
                if n[r] == 0:
                    continue
                mine = slice(first[r], first[r] + n[r])
                pos = host.length(r) + np.arange(n[r])
                z = OC.rotate(OC.norm(x[mine, Hq:Hq + Hkv], w[1], 1e-6), pos, freq, False)
                val = x[mine, Hq + Hkv:]
                top = np.abs(z).reshape(*z.shape[:-1], -1, 32).max(-1).repeat(32, -1)
                kd, vd = kr[r, :n[r]], vr[r, :n[r]]
                if fmt == BF16:
                    assert np.all(np.abs(kd - z) <= HALF * np.abs(z) + 64 * F32 * 2 * np.abs(z).max())
                    assert np.array_equal(vd, val)
                else:
                    # half of the widest step (4 to 6), or 7 to 6, is one unit 2^e, and top > 3.5 * 2^e
                    assert np.all(np.abs(kd - z) <= top * (2 / 7) * (1 + 2.0 ** -20))
                    assert np.array_equal(kd, OC.quantise_k(kd))
                    q4 = OC.quantise_v(val)
                    assert np.all(np.abs(vd - q4) <= HALF * np.abs(q4) * (1 + HALF))
                check_attention(o[mine], qn[mine], *dense[r], pos, scale, window, sinks, fmt)
            assert np.all(o[0] == 5.0) and np.all(o[-1] == 5.0)
            after.append(dense)
        acc = rng.integers(0, gamma + 1, R)
        c.commit(torch.tensor(acc, dtype=torch.int32, device=dev))
        for r in range(R):
            if n[r]:
                keep = host.length(r) + min(acc[r], n[r] - 1) + 1
                host.kv[r] = [(after[i][r][0][:keep], after[i][r][1][:keep]) for i in range(layers)]
        assert c.length.cpu().tolist() == [host.length(r) for r in range(R)]
        if step % 2 == 0:
            parent = np.arange(R)
            parent[rng.integers(0, R, 2)] = rng.integers(-1, R, 2)
            if step == 4:
                parent = rng.permutation(R)
            c.fork(torch.tensor(parent, dtype=torch.int32, device=dev))
            host.fork(parent)
        if step % 3 == 2:
            c.compact()
            used = int((c.ref > 0).sum())
            assert bool((c.ref[:used] > 0).all())
        T = max(1, max(host.length(r) for r in range(R)))
        for layer in range(layers):
            k, v = c.read(layer, T)
            k, v = back(k), back(v)
            for r in range(R):
                m = host.length(r)
                lo = max(0, m - window + 1) if window else 0  # the rest may have been released
                assert np.array_equal(k[r, lo:m], host.kv[r][layer][0][lo:])
                assert np.array_equal(v[r, lo:m], host.kv[r][layer][1][lo:])
                assert np.array_equal(k[r, :min(m, sinks)], host.kv[r][layer][0][:sinks])


class Target:
    """One attention layer over the cache as a round's target, deterministic
    and with nothing allocated that outlives a call."""

    def __init__(self, d, Hq, Hkv, D, dev):
        g = torch.Generator().manual_seed(5)
        self.emb = torch.randn((d.V, Hq + 2 * Hkv, D), generator=g).to(torch.bfloat16).to(dev)
        self.head = (torch.randn((Hq * D, d.V), generator=g) * 0.5).to(dev)
        self.freq = (1e4 ** (-2.0 * torch.arange(D // 2, dtype=torch.float64) / D)).to(dev)
        self.Hq, self.Hkv = Hq, Hkv

    def __call__(self, d, cache, ell):
        tok = torch.cat([d.x0.view(-1, 1), d.x], dim=1).view(-1).long()
        x = self.emb[tok]
        Hq, Hkv = self.Hq, self.Hkv
        q = cache.append(0, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], freq=self.freq)
        self.out = torch.zeros_like(q)
        cache.attend(0, q, out=self.out)
        self.q = q
        d.target.copy_((self.out.view(q.shape[0], -1).float() @ self.head).view(d.target.shape))


def test_run_round_cached(dev):
    """Three rounds of the whole path: what is verified is what the target
    computed, the cache grows by the accepted rows, and the attention of
    every round is the oracle's over all tokens accepted before."""
    from semi_ar_draft_round_amd import device_round as DR
    from semi_ar_draft_round_amd.cache import PagedCache
    w = W.custom("cached_r5_g6_v500", R=5, gamma=6, V=500, r=32, d=64, dtype="f32", seed=71)
    Hq, Hkv, D = 4, 2, 64
    c = PagedCache(1, w.R, 200, 80, Hkv, D, page=16)
    host = Host(c, w.R, 1, Hkv, D)
    target = None
    x0 = None
    for rnd in range(3):
        d = DR.to_device(W.make_inputs(w, round_index=rnd), dev)
        target = target or Target(d, Hq, Hkv, D, dev)
        if x0 is not None:
            d.x0.copy_(x0)
        before = c.length.cpu().tolist()
        dense = []

        def forward(d, cache, ell):
            target(d, cache, ell)
            dense.append(host.take_rows(0, ell.cpu(), w.gamma)[0])

        DR.run_round_cached(d, c, forward)
        out = DR.outputs_to_host(d)
        n_acc, next_tok = out["n_acc"].tolist(), out["next_tok"].tolist()
        ell = c.ell.cpu().tolist()
        assert ell == out["ell"].tolist()
        o, q = back(target.out), back(target.q)
        for r in range(w.R):
            f, n = r * (w.gamma + 1), ell[r] + 1
            pos = before[r] + np.arange(n)
            check_attention(o[f:f + n], q[f:f + n], *dense[0][r], pos, D ** -0.5, 0, 0, BF16)
            keep = before[r] + min(n_acc[r], ell[r]) + 1
            host.kv[r] = [(dense[0][r][0][:keep], dense[0][r][1][:keep])]
        assert c.length.cpu().tolist() == [host.length(r) for r in range(w.R)]
        DR.run_round(d)                       # the target's logits given: the same round
        again = DR.outputs_to_host(d)
        assert again["n_acc"].tolist() == n_acc and again["next_tok"].tolist() == next_tok
        x0 = d.next_tok.clone()
    assert sum(host.length(r) for r in range(w.R)) >= 3 * w.R


@pytest.mark.parametrize("fmt", [BF16, FP4])
def test_captured_round_of_the_whole_path(fmt, dev):
    """One graph of a round with its cache, replayed with eager work and
    synchronizations between: after every replay the state equals that of the
    same rounds run eagerly."""
    from semi_ar_draft_round_amd import device_round as DR
    from semi_ar_draft_round_amd.cache import PagedCache
    w = W.custom("captured_r7_g5_v400", R=7, gamma=5, V=400, r=32, d=64, dtype="f32", seed=72)
    Hq, Hkv, D = 4, 2, 64
    ds = [DR.to_device(W.make_inputs(w), dev) for _ in range(2)]
    cs = [PagedCache(1, w.R, 120, 60, Hkv, D, page=16, fmt=fmt, window=48, sinks=2) for _ in range(2)]
    ts = [Target(d, Hq, Hkv, D, dev) for d in ds]

    def step(i):
        DR.run_round_cached(ds[i], cs[i], ts[i])
        ds[i].x0.copy_(ds[i].next_tok)

    for i in range(2):
        cs[i].pool.zero_()
    x0 = ds[0].x0.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(1)                                               # warm up, then start again
    torch.cuda.synchronize()
    cs[1].reset()
    cs[1].pool.zero_()
    ds[1].x0.copy_(x0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(1)
    for rep in range(5):
        say(f"[round] replay {rep}")
        g.replay()
        torch.cuda.synchronize()
        step(0)
        torch.cuda.synchronize()
        for name in ("table", "length", "ref", "bits", "ell", "pool"):
            assert torch.equal(getattr(cs[0], name), getattr(cs[1], name)), (rep, name)
        for name in ("x", "n_acc", "next_tok", "target"):
            assert torch.equal(getattr(ds[0], name), getattr(ds[1], name)), (rep, name)


def test_a_request_without_pages_keeps_its_cache(dev):
    """Refused requests (ell -1) change nothing, their rows are not written,
    and the others' round goes on."""
    from semi_ar_draft_round_amd import binding as B
    from semi_ar_draft_round_amd.cache import PagedCache
    c = PagedCache(1, 3, 64, 5, 1, 64, page=16)
    g = torch.Generator().manual_seed(9)
    x = torch.randn((3 * 17, 3, 64), generator=g).to(torch.bfloat16).to(dev)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)
    assert c.reserve(i32(15, 15, 15), 16).tolist() == [15, 15, 15]
    c.append(0, x[:, :1], x[:, 1:2], x[:, 2:])
    c.commit(i32(15, 15, 15))
    k0, v0 = c.read(0, 16)
    assert c.reserve(i32(16, 0, 0), 16).tolist() == [16, -1, -1]
    assert int(c.status) == B.ENOPAGES
    q = c.append(0, x[:, :1], x[:, 1:2], x[:, 2:], q_out=torch.full((51, 1, 64), 3.0, dtype=torch.bfloat16, device=dev))
    out, _ = c.attend(0, q, out=torch.full((51, 1, 64), 3.0, dtype=torch.bfloat16, device=dev))
    assert bool((q[17:] == 3).all()) and bool((out[17:] == 3).all()) and not bool((out[:17] == 3).all())
    c.commit(i32(16, 16, 16))
    assert c.length.tolist() == [33, 16, 16]
    k1, v1 = c.read(0, 16)
    assert torch.equal(k0, k1) and torch.equal(v0, v1)
