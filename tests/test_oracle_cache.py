"""The cache oracle against properties of its own: page layouts round-trip,
the 4-bit rounding is the nearest value, attention reduces to known cases."""

import numpy as np
import pytest

from oracle import cache as OC
from cache_cases import BF16, FP4, bf, make_tokens, page_bytes


def test_quantise_v_is_nearest():
    rng = np.random.default_rng(1)
    _, v = bf(rng.standard_normal((50, 3, 64)))
    y = OC.quantise_v(v)
    unit = np.abs(v).max(-1, keepdims=True) / 6
    grid = np.concatenate([-OC.E2M1[::-1], OC.E2M1])
    best = np.abs(v[..., None] / unit[..., None] - grid).min(-1)
    assert np.all(np.abs(v / unit - y / unit) <= best + 1e-6)
    assert np.all(OC.quantise_v(np.zeros((1, 1, 64))) == 0)
    bad = v[:1, :1].copy()
    bad[..., 5] = np.inf
    assert np.isnan(OC.quantise_v(bad)).all()


def test_quantise_k_is_nearest_and_unsaturated():
    rng = np.random.default_rng(2)
    k = rng.standard_normal((40, 2, 64)) * np.exp2(rng.integers(-20, 20, (40, 2, 1)))
    y = OC.quantise_k(k)
    g, z = k.reshape(40, 2, 2, 32), y.reshape(40, 2, 2, 32)
    top = np.abs(g).max(-1, keepdims=True)
    e = np.floor(np.log2(top)) - 2
    e = np.where(top / np.exp2(e) > 7, e + 1, e)
    assert np.all(np.abs(g - z) <= np.exp2(e))       # half of the last step (2 units)
    # half-way values go to the even code
    x = np.zeros((1, 1, 32))
    x[0, 0, :8] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25]
    assert OC.quantise_k(x)[0, 0, :8].tolist() == [6, 4, 4, 2, 2, 1, 1, 0]
    x[0, 0, 0] = 7.0
    assert OC.quantise_k(x)[0, 0, 0] == 6
    x[0, 0, 0] = 7.01
    assert OC.quantise_k(x)[0, 0, 0] == 8


@pytest.mark.parametrize("fmt", [BF16, FP4])
def test_pages_hold_every_value_once(fmt):
    """Every value of a page lands in bytes of its own: two fills that differ
    in one value differ in that value's bytes only."""
    rng = np.random.default_rng(3)
    H, D, P, T = 2, 64, 32, 40
    table = np.array([2, 0])
    k, v, _, _ = make_tokens(rng, fmt, T, H, D)
    pool = np.zeros((3, page_bytes(fmt, H, D, P)), dtype=np.uint8)
    OC.write_pages(fmt, k, v, table, P, pool)
    assert not pool[1].any()
    other = pool.copy()
    kc = k if fmt == BF16 else k[0]
    kc[33, 1, 17] ^= 1
    OC.write_pages(fmt, k, v, table, P, other)
    diff = np.argwhere(pool != other)
    assert len(diff) == 1 and diff[0, 0] == 0
    if fmt == BF16:   # [head][K][block][D/8][16 tokens][8 dims]
        assert diff[0, 1] // 2 == (P * 2 * D) + (17 // 8 * 16 + 1) * 8 + 17 % 8


def test_attention_one_visible_token_is_its_value():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((3, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    o, lse = OC.attention(q, k, v, [4, 5, 8], 0.3, 1, 0)
    for i, p in enumerate((4, 5, 8)):
        for h in range(4):
            assert np.allclose(o[i, h], v[p, h // 2])
            assert np.isclose(lse[i, h], k[p, h // 2] @ q[i, h] * 0.3)
    o, lse = OC.attention(q, k, v, [4, 5, 8], 0.3, 0, 0, have=np.zeros(9, bool))
    assert not o.any() and np.isneginf(lse).all()


def test_rotation_depends_on_the_distance_only():
    rng = np.random.default_rng(5)
    f = 1e4 ** (-np.arange(4) / 4)
    for adjacent in (False, True):
        a, b = rng.standard_normal((1, 1, 10)), rng.standard_normal((1, 1, 10))
        dot = lambda p, s: (OC.rotate(a, [p], f, adjacent) * OC.rotate(b, [s], f, adjacent)).sum()
        assert np.isclose(dot(7, 3), dot(107, 103))
        assert np.allclose(OC.rotate(a, [0], f, adjacent), a)


def test_pages_fork_and_copy_on_write():
    p = OC.Pages(4, 8, 4, 16)
    assert p.reserve([4, -1, -1, -1], 8) == ([4, -1, -1, -1], [], False)
    p.commit([4, -1, -1, -1], [9, 0, 0, 0], 8, 0, 0)
    assert p.len.tolist() == [5, 0, 0, 0] and p.table[0, 0] == 0
    p.fork([0, 0, 0, 3])
    assert p.refs()[0] == 3 and p.len.tolist() == [5, 5, 5, 0]
    out, pairs, refused = p.reserve([0, 0, 0, -1], 8)
    assert out == [0, 0, 0, -1] and pairs == [(0, 1), (0, 2)] and not refused   # the last holder keeps page 0
    assert p.table[:3, 0].tolist() == [1, 2, 0]
    p.fork([-1, 0, 2, 3])
    assert p.len.tolist() == [0, 5, 5, 0]
    assert p.compact() == [] and sorted(p.table[1:3, 0].tolist()) == [0, 1]
