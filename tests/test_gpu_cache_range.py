"""The paged cache's operators at the ends of the values' range: what a plain
softmax or norm in the same types gives has to come out, without infinities of
its own."""

import sys

import numpy as np
import pytest

from cache_cases import BF16, F32, FP4, HALF, attention_tolerance, bf, page_bytes
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


def one_request(fmt, k, v, P):
    """A pool of one request's tokens and its table.  k, v: what write_pages takes."""
    codes = k if fmt == BF16 else k[0]
    T, H, D = codes.shape
    n = -(-T // P)
    pool = np.full((n + 1, page_bytes(fmt, H, D, P)), 0xFF, dtype=np.uint8)
    table = np.random.default_rng(0).permutation(n + 1)[:n].astype(np.int32)
    OC.write_pages(fmt, k, v, table, P, pool)
    return pool, table[None]


def attend(dev, fmt, pool, table, q, first, P, heads_kv):
    """q [rows][Hq][D] bits at positions first ..; float64 out and lse."""
    from semi_ar_draft_round_amd import binding as B
    rows = q.shape[0]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
    lse = torch.zeros(q.shape[:2], dtype=torch.float32, device=dev)
    out, _ = B.dspark_cache_attention(t16(q, dev), torch.from_numpy(pool).to(dev), torch.from_numpy(table).to(dev),
                                      i32(first), i32(rows - 1), rows - 1, fmt=fmt, page=P, heads_kv=heads_kv, lse=lse)
    return back(out), lse.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("power", [115, -90])
def test_values_far_from_one(power, D, fmt, dev):
    """Values near 2^power.  16 tokens x 8 query heads fill four row tiles, so
    a wave goes through tiles in turn; the first has scores of 0, the others
    of 5.3, and in every fourth row of -5.3 (2^7.65 and 2^-7.65): less than
    8 ln 2 above the first.  |v| adds up to less than 300 * 6 * 2^115 < 2^126,
    which the header allows; weights relative to the first tile's maximum
    would reach 2^7.6 and 32 of them times 2^116 overflow.  At 2^-90 weights
    are above 2^-24, so that their product with a scale is a normal number.

    The bound is attention_tolerance's for the values divided by 2^power, a
    power of two, so every relative rounding is the same."""
    say(f"[range] attention fmt {fmt} D {D} 2^{power}")
    rng = np.random.default_rng(D + fmt)
    T, rows, Hq, P = 300, 16, 8, 32
    late = np.arange(T) >= 32
    if fmt == BF16:
        kb, k = bf(np.where(late, 0.5, 0.0)[:, None, None] * np.ones((T, 1, D)))
        vb, v = bf(rng.uniform(1, 4, (T, 1, D)))
        stored = bf(v * 2.0 ** power)[0]
        pool, table = one_request(fmt, kb, stored, P)
    else:
        kc = np.where(late, 2, 0)[:, None, None].astype(np.uint8) * np.ones((1, 1, D), np.uint8)
        kb = np.full((T, 1, D // 32), 126, np.uint8)
        vc = rng.integers(2, 8, (T, 1, D)).astype(np.uint8)
        vs = rng.uniform(0.25, 1, (T, 1)).astype(np.float32)
        k, v = OC.E2M1[kc] * 0.5, OC.E2M1[vc] * vs.astype(np.float64)[..., None]
        pool, table = one_request(fmt, (kc, kb), (vc, vs * np.float32(2.0 ** power)), P)
    a = {64: 1.328125, 128: 0.9375, 256: 0.6640625}[D]
    qb, q = bf(np.where(np.arange(rows) % 4 == 3, -a, a)[:, None, None] * np.ones((rows, Hq, D)))
    pos = T - rows + np.arange(rows)
    o, lse = attend(dev, fmt, pool, table, qb, T - rows, P, 1)
    want, wz = OC.attention(q, k, v, pos, D ** -0.5, 0, 0)
    tol, tz = attention_tolerance(q, k, v, pos, D ** -0.5, 0, 0, want)
    assert np.isfinite(o).all()
    err = np.abs(o / 2.0 ** power - want)
    assert np.all(err <= tol), float((err / tol).max())
    assert np.all(np.abs(lse - wz) <= tz + 2.0 ** -22 * np.abs(wz))


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norms_of_large_and_small_heads(eps, D, fmt, dev):
    """Rows of every magnitude that bf16 has, side by side: the square of
    2^100 is past fp32's range and that of 2^-100 below it, the norm is not.
    The bound is the append's: 32 roundings of fp32 doubled, then half a step
    of bf16.  A 4-bit key is off by at most one unit 2^e, top > 3.5 * 2^e."""
    from semi_ar_draft_round_amd import binding as B
    say(f"[range] norms fmt {fmt} D {D} eps {eps}")
    rng = np.random.default_rng(D)
    power = np.array([0, 59, 60, 61, 62, 63, 64, 100, 127, -1, -47, -48, -49, -62, -64, -74, -100, -120, 0, 127])
    rows, Hq, Hkv, P = len(power), 3, 2, 32
    x = rng.uniform(0.25, 1, (rows, Hq + 2 * Hkv, D)) * rng.choice([-1, 1], (rows, Hq + 2 * Hkv, D))
    xb, x = bf(x * 2.0 ** power[:, None, None])
    wb, w = bf(1 + 0.3 * rng.standard_normal((2, D)))
    xt = t16(xb, dev)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)
    pool = torch.full((2, B.dspark_cache_page_bytes(fmt, Hkv, D, P)), 255, dtype=torch.uint8, device=dev)
    table = i32(1, 0).view(1, 2)
    q = B.dspark_cache_append(xt[:, :Hq], xt[:, Hq:Hq + Hkv], xt[:, Hq + Hkv:], pool, table, i32(0), i32(rows - 1),
                              rows - 1, fmt=fmt, page=P, wq=t16(wb[0], dev), wk=t16(wb[1], dev), eps=eps)
    k, _ = B.dspark_cache_read(pool, table, None, i32(rows), rows, fmt=fmt, page=P, heads_kv=Hkv, dim=D)
    z = OC.norm(x[:, :Hq], w[0], eps)
    assert np.all(np.abs(back(q) - z) <= (HALF + 64 * F32) * np.abs(z) + 2.0 ** -134)
    z, kd = OC.norm(x[:, Hq:Hq + Hkv], w[1], eps), back(k)[0]
    if fmt == BF16:
        assert np.all(np.abs(kd - z) <= (HALF + 64 * F32) * np.abs(z) + 2.0 ** -134)
    else:
        top = np.abs(z).reshape(rows, Hkv, -1, 32).max(-1).repeat(32, -1)
        assert np.all(np.abs(kd - z) <= np.maximum(top * (2 / 7) * (1 + 2.0 ** -20), 2.0 ** -126))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_every_key_scale_reads_back(D, dev):
    """Tokens whose K scale bytes go through 0 (2^-127), 1 .. 252 and 255
    (NaN): the values that the header names, exactly."""
    from semi_ar_draft_round_amd import binding as B
    say(f"[range] scales read D {D}")
    rng = np.random.default_rng(D)
    scale = np.concatenate([np.arange(253), [255, 0, 255]])
    T, E, P = len(scale), D // 32, 64
    kc = rng.integers(0, 16, (T, 1, D)).astype(np.uint8)
    kb = np.stack([np.roll(scale, i) for i in range(E)], -1)[:, None].astype(np.uint8)
    pool, table = one_request(FP4, (kc, kb), (kc, np.ones((T, 1), np.float32)), P)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)
    k, _ = B.dspark_cache_read(torch.from_numpy(pool).to(dev), torch.from_numpy(table).to(dev), None, i32(T), T, fmt=FP4,
                               page=P, heads_kv=1, dim=D)
    s = np.repeat(np.where(kb == 255, np.nan, 2.0 ** (kb.astype(np.float64) - 127)), 32, axis=-1)
    assert np.array_equal(back(k)[0], np.where(kc & 8, -1.0, 1.0) * OC.E2M1[kc & 7] * s, equal_nan=True)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt,byte", [(FP4, 0), (FP4, 1), (FP4, 20), (FP4, 234), (FP4, 252), (BF16, 0), (BF16, 252)])
def test_keys_far_from_one(fmt, byte, D, dev):
    """Visible keys whose scale is 2^(byte - 127), the smallest ones subnormal
    in bf16, against queries that bring the scores back to the order of one."""
    say(f"[range] keys fmt {fmt} byte {byte} D {D}")
    rng = np.random.default_rng(D + byte)
    T, rows, Hq, P = 70, 6, 4, 32
    kc = rng.integers(0, 16, (T, 1, D)).astype(np.uint8)
    k = np.where(kc & 8, -1.0, 1.0) * OC.E2M1[kc & 7] * 2.0 ** (byte - 127)
    if fmt == FP4:
        vc, vs = rng.integers(0, 16, (T, 1, D)).astype(np.uint8), rng.uniform(0.1, 0.6, (T, 1)).astype(np.float32)
        v = np.where(vc & 8, -1.0, 1.0) * OC.E2M1[vc & 7] * vs.astype(np.float64)[..., None]
        pool, table = one_request(FP4, (kc, np.full((T, 1, D // 32), byte, np.uint8)), (vc, vs), P)
    else:
        vb, v = bf(rng.standard_normal((T, 1, D)))
        kb, same = bf(k)
        assert np.array_equal(same, k)
        pool, table = one_request(BF16, kb, vb, P)
    qb, q = bf(rng.uniform(0.25, 1, (rows, Hq, D)) * rng.choice([-1, 1], (rows, Hq, D)) * 2.0 ** min(126, 126 - byte))
    pos = T - rows + np.arange(rows)
    o, lse = attend(dev, fmt, pool, table, qb, T - rows, P, 1)
    want, wz = OC.attention(q, k, v, pos, D ** -0.5, 0, 0)
    tol, tz = attention_tolerance(q, k, v, pos, D ** -0.5, 0, 0, want)
    err = np.abs(o - want)
    assert np.all(err <= tol), float((err / tol).max())
    assert np.all(np.abs(lse - wz) <= tz + 2.0 ** -22 * np.abs(wz))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_visible_nan_scales(D, dev):
    """A NaN scale of a visible key makes the rows that see it NaN, of a
    visible value too, and leaves the other rows alone."""
    say(f"[range] NaN scales D {D}")
    rng = np.random.default_rng(D)
    T, rows, P = 70, 6, 32
    for what in ("key", "value"):
        kc, vc = (rng.integers(0, 16, (T, 2, D)).astype(np.uint8) for _ in range(2))
        kb, vs = rng.integers(123, 127, (T, 2, D // 32)).astype(np.uint8), rng.uniform(0.1, 0.6, (T, 2)).astype(np.float32)
        if what == "key":
            kb[T - 3, 1, D // 32 - 1] = 255
        else:
            vs[T - 3, 1] = np.nan
        pool, table = one_request(FP4, (kc, kb), (vc, vs), P)
        qb, q = bf(rng.standard_normal((rows, 4, D)))
        o, lse = attend(dev, FP4, pool, table, qb, T - rows, P, 2)
        sees = np.zeros((rows, 4), dtype=bool)
        sees[3:, 2:] = True                            # positions T - 3 .. of the heads that read head 1
        assert np.array_equal(np.isnan(o).all(-1), sees) and np.array_equal(np.isnan(o).any(-1), sees)
        assert np.array_equal(np.isnan(lse), sees if what == "key" else np.zeros_like(sees))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows,Hq", [(1, 1), (5, 8), (16, 8)])
def test_infinities_that_every_row_sees(rows, Hq, D, dev):
    """Infinite values of tokens far below every row's position, where no tile
    needs a mask: they come out as infinities with their sign, two of unlike
    sign in a dim as NaN, and every other dim as if they were not there."""
    say(f"[range] infinities D {D} rows {rows}")
    rng = np.random.default_rng(D + rows)
    T, P = 700, 32
    kb, k = bf(rng.standard_normal((T, 1, D)))
    vb, v = bf(rng.standard_normal((T, 1, D)))
    v[40, 0, 3] = v[41, 0, 3] = v[300, 0, 3] = np.inf
    v[41, 0, 7] = -np.inf
    v[130, 0, D - 1] = -np.inf
    v[333, 0, 20], v[500, 0, 20] = np.inf, -np.inf
    vb[~np.isfinite(v)] = np.where(v[~np.isfinite(v)] > 0, 0x7F80, 0xFF80)
    pool, table = one_request(BF16, kb, vb, P)
    qb, q = bf(rng.standard_normal((rows, Hq, D)))
    pos = T - rows + np.arange(rows)
    o, _ = attend(dev, BF16, pool, table, qb, T - rows, P, 1)
    with np.errstate(invalid="ignore"):
        want, _ = OC.attention(q, k, v, pos, D ** -0.5, 0, 0)
    assert np.array_equal(np.isnan(o), np.isnan(want)) and np.isnan(want[..., 20]).all()
    assert np.array_equal(np.isposinf(o), np.isposinf(want)) and np.isposinf(want[..., 3]).all()
    assert np.array_equal(np.isneginf(o), np.isneginf(want)) and np.isneginf(want[..., [7, D - 1]]).all()
    fine = np.isfinite(want)
    tol, _ = attention_tolerance(q, k, v, pos, D ** -0.5, 0, 0, np.where(fine, want, 0))
    assert np.all(np.abs(np.where(fine, o, 0) - np.where(fine, want, 0)) <= np.where(fine, tol, 0))
