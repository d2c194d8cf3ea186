"""dspark_verify over rows with tokens of no mass (a grammar's mask, a bias of
-inf): none of them is ever drawn, wherever u_res falls.

The draw adds up the masses of chunks of 16 tokens, a run of chunks a thread.
u_res is set beside every border between two threads' runs, where the sums of
either side differ by roundings, on rows whose runs and chunks begin with
tokens of no mass."""

import sys

import numpy as np
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


def masked_row(V, dtype, seed):
    """One row's logits as stored and what is allowed: of every chunk all but its
    first tokens and some others, of every 16 chunks all but the first."""
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((rng.standard_normal(V) * 2).astype(np.float32)).to(dtype)
    v = np.arange(V)
    allowed = (v % 16 >= 1 + rng.integers(0, 8, -(-V // 16))[v // 16]) & (rng.random(V) < 0.7) & (v // 16 % 16 != 0)
    x[torch.from_numpy(~allowed)] = -float("inf")
    return x, allowed


def draw(dev, row, u, admitted=0, **kw):
    """next_tok of len(u) requests that all have the same target rows (`row`, as
    often as one with `admitted` drafts has), none of whose drafts is accepted."""
    from semi_ar_draft_round_amd import binding as B
    R, V = len(u), row.shape[0]
    i32 = dict(dtype=torch.int32, device=dev)
    U = kw.pop("U", None)
    U = torch.zeros((R, 1, V), dtype=row.dtype, device=dev) if U is None else U
    W = torch.zeros((V, 32), dtype=row.dtype, device=dev)
    one = lambda x: torch.full((R, 1), x, dtype=torch.float32, device=dev)
    target = row.to(dev)[None].expand(admitted + 1, V).contiguous()
    n, tok = B.dspark_verify(target, U, W, W, torch.zeros(R, **i32), torch.ones((R, 1), **i32), kw.pop("lse", one(0.0)),
                             kw.pop("logit", one(0.0)), torch.full((R,), admitted, **i32), one(1.0),
                             torch.from_numpy(u).to(dev), row0=torch.zeros(R, **i32))
    torch.cuda.synchronize()
    assert not n.any()
    return tok.cpu().numpy()


@pytest.mark.parametrize("V,dtype", [(16384, torch.bfloat16), (16384, torch.float32), (50257, torch.float32),
                                     (129280, torch.bfloat16), (151936, torch.bfloat16), (200003, torch.bfloat16)])
def test_borders_between_threads(V, dtype, dev):
    say(f"[verify] borders {V} {dtype}")
    row, allowed = masked_row(V, dtype, V)
    x = row.double().numpy()
    p = np.exp(x - x[allowed].max())
    cdf = np.cumsum(p) / p.sum()
    run = -(-(-(-V // 64)) // 256) * 64                      # tokens of a thread
    borders = np.arange(run, V, run)
    borders = borders[cdf[borders - 1] > 0.02]
    # fp32 sums of these masses are within some 1e-6 of the exact ones
    far = 64
    step = np.arange(-far, far + 1)
    centre = cdf[borders - 1].astype(np.float32).view(np.int32)
    u = (centre[:, None] + step[None]).reshape(-1).view(np.float32)
    u = np.concatenate([u, np.float32([0, 2.0 ** -149, 1e-7, 1 - 2.0 ** -24, 1 - 2.0 ** -23])])
    u = np.clip(u, np.float32(0), np.float32(1 - 2.0 ** -24))
    bad, R = 0, 1024
    U = torch.zeros((R, 1, V), dtype=dtype, device=dev)
    for at in range(0, len(u), R):
        part = u[at:at + R]
        tok = draw(dev, row, part, U=U[:len(part)])
        assert np.all((tok >= 0) & (tok < V))
        bad += int((~allowed[tok]).sum())
        lo = np.where(tok > 0, cdf[np.maximum(tok, 1) - 1], 0)
        assert np.all((part >= lo - 1e-5) & (part <= cdf[tok] + 1e-5))
    say(f"  {len(u)} draws, {bad} of a forbidden token")
    assert bad == 0


@pytest.mark.parametrize("V,dtype", [(16384, torch.bfloat16), (20000, torch.float32), (129280, torch.bfloat16)])
def test_a_residual_of_roundings(V, dtype, dev):
    """Target and draft alike but for the last bits of the draft's log-sum: what
    is left of a chunk is rounding, and which of its tokens have some differs
    between the sums and the draw."""
    say(f"[verify] roundings {V} {dtype}")
    rng = np.random.default_rng(V)
    x = torch.from_numpy((rng.standard_normal(V) * 2).astype(np.float32)).to(dtype)
    # one token allowed in a chunk, never its first
    allowed = np.zeros(-(-V // 16) * 16, bool)
    allowed[np.arange(0, len(allowed), 16) + rng.integers(1, 16, len(allowed) // 16)] = True
    allowed = allowed[:V]
    row = x.clone()
    row[torch.from_numpy(~allowed)] = -float("inf")
    z = np.float32(torch.logsumexp(row.double(), 0).item())
    R = 2048
    U = row.to(dev)[None, None].expand(R, 1, V).contiguous()
    lse = (np.full(R, z).view(np.int32) + np.arange(R) % 4 - 1).astype(np.int32).view(np.float32)
    u = ((np.arange(R) + 0.5) / R).astype(np.float32)
    tok = draw(dev, row, u, admitted=1, U=U, lse=torch.from_numpy(lse)[:, None].contiguous().to(dev),
               logit=torch.full((R, 1), 1e4, device=dev))
    bad = int((~allowed[tok]).sum())
    say(f"  {len(u)} draws, {bad} of a forbidden token")
    assert bad == 0


@pytest.mark.parametrize("V,dtype", [(16384, torch.bfloat16), (20003, torch.float32)])
def test_rows_that_allow_one_token_or_none(V, dtype, dev):
    say(f"[verify] one token {V} {dtype}")
    u = np.float32([0, 1e-6, 0.3, 0.99, 1 - 2.0 ** -24])
    for only in (0, 1, 15, 16, 63, 64, V // 2 + 7, V - 1):
        row = torch.full((V,), -float("inf")).to(dtype)
        row[only] = -3.0
        assert np.all(draw(dev, row, u) == only)
    tok = draw(dev, torch.full((V,), -float("inf")).to(dtype), u)
    assert np.all((tok >= 0) & (tok < V))


@pytest.mark.parametrize("w", [dict(R=130, gamma=4, V=4096, r=256, d=128), dict(R=70, gamma=6, V=4100, r=64, d=128),
                               dict(R=20, gamma=5, V=1000, r=32, d=64), dict(R=40, gamma=7, V=336, r=20, d=36, dtype="f32")],
                         ids=lambda w: f"V{w['V']}")
def test_masked_rounds_against_oracle(w, dev):
    """Drafts some of which a mask rules out, accepted and drawn as the oracle
    does, from rows that dspark_logits has masked; greedily too."""
    from oracle import verify as OV
    from oracle.common import as_f64
    from parity import check_verify
    from semi_ar_draft_round_amd import binding as B
    from semi_ar_draft_round_amd import device_round as DR
    from semi_ar_draft_round_amd import workloads as W
    say(f"[verify] masked rounds {w}")
    rng = np.random.default_rng(w["V"])
    inp = W.make_inputs(W.custom("masked", seed=71, **w))
    d = DR.to_device(inp, dev)
    DR.sample_conf(d)
    d.ell.copy_(torch.from_numpy(rng.integers(0, w["gamma"] + 1, w["R"]).astype(np.int32)))
    x = d.x.cpu().numpy()
    R, g1, V = d.target.shape
    allowed = rng.random((R, g1, V)) < rng.choice([0.03, 0.5, 0.9], (R, g1, 1))
    r, i = np.mgrid[:R, :g1 - 1]
    allowed[r, i, x] = rng.random((R, g1 - 1)) < 0.8
    allowed[..., V - 1] = True
    bits = np.zeros((R * g1, -(-V // 32) * 32), bool)
    bits[:, :V] = allowed.reshape(R * g1, V)
    mask = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32)).to(dev)
    B.dspark_logits(d.target, None, d.ell, w["gamma"], None, mask=mask, out=d.target)
    DR.verify(d)
    DR.verify_greedy(d)
    out = DR.outputs_to_host(d)
    # -1e4: no mass either, and finite for the bounds
    target = np.where(allowed, as_f64(inp.target, inp.w.dtype), -1e4)
    rep = check_verify(inp, dict(out, ell=d.ell.cpu().numpy()), np.arange(R), target=target)
    n, tok = out["n_acc"], out["next_tok"]
    assert all(allowed[q, k, x[q, k]] for q in range(R) for k in range(n[q])) and allowed[np.arange(R), n, tok].all()
    assert n.max() >= 2
    want = OV.verify_greedy(target, None, x, d.ell.cpu().numpy())
    assert np.array_equal(want["n_acc"], d.n_acc_g.cpu().numpy())
    assert np.array_equal(want["next_tok"], d.next_tok_g.cpu().numpy())
    say(f"  {rep}, up to {n.max()} accepted")
