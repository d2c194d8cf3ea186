"""The cache's operators over declared blocks that are much larger than what
most requests bring: prompts beside single tokens, idle slots, the largest
block; and rotations of a part of a head.  Bounds as in
test_gpu_cache_attention.py and test_gpu_cache_append.py."""

import sys

import numpy as np
import pytest

from cache_cases import BF16, F32, FP4, HALF, bf
from oracle import cache as OC
from test_gpu_cache_attention import Case, back, dev, say, t16  # noqa: F401  (dev: a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def spread(R, live):
    """lens and ells of R slots: those of `live` (slot: (len, ell)), the others idle or as live[None] says."""
    other = live.get(None)
    lens = [live[r][0] if r in live else other[0](r) if other else 0 for r in range(R)]
    return lens, [live[r][1] if r in live else other[1] if other else -1 for r in range(R)]


# name: R, {slot: (len, ell), None: (len of r, ell)}, Hq, Hkv, D, P, gamma, window, sinks
MIXED = {
    # a chunk beside single tokens: 300 x 19 row blocks declared, 318 with rows
    "chunk": (300, {150: (33, 299), None: (lambda r: 3 + 7 * r % 40, 0)}, 8, 1, 64, 32, 299, 0, 0),
    "chunk-window": (270, {0: (70, 200), 269: (5, 190), None: (lambda r: 1 + 11 * r % 60, 0)}, 8, 1, 128, 16, 200, 40, 3),
    # ragged blocks: some requests have one row block, some several, some none
    "ragged": (130, {r: (r % 50, [-1, 0, 20, 60][r % 4]) for r in range(130)}, 8, 1, 64, 16, 60, 0, 0),
    # few live slots of very unequal length, runs of units cross the idle ones
    "idle-128": (128, {0: (9000, 16), 61: (50, 16), 127: (700, 3)}, 8, 8, 64, 64, 16, 0, 0),
    "idle-1000": (1000, {3: (40, 16), 500: (6000, 16), 501: (30, 0), 999: (700, 16)}, 8, 8, 64, 64, 16, 0, 0),
    "last": (4096, {4095: (100, 2)}, 4, 2, 128, 64, 2, 0, 0),
    "nobody": (4096, {}, 4, 2, 128, 64, 2, 0, 0),
    # more heads on a head than a row block has rows
    "wide": (7, {2: (20, 3), 5: (64, 1), 6: (0, 0)}, 300, 1, 64, 16, 200, 0, 0),
}


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("name", MIXED)
def test_attention_of_mixed_blocks(name, fmt, dev):
    R, live, Hq, Hkv, D, P, gamma, window, sinks = MIXED[name]
    say(f"[blocks] {name} fmt {fmt}")
    lens, ells = spread(R, live)
    Case(dev, fmt, lens, ells, Hq, Hkv, D, P, gamma, window, sinks, seed=30).check()


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5)])
def test_attention_of_the_largest_block(window, sinks, fmt, dev):
    say(f"[blocks] 1024 rows fmt {fmt} window {window}")
    Case(dev, fmt, [70, 0], [1023, 5], 4, 2, 64, 64, 1023, window, sinks, seed=31).check()


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("D,rot,adjacent", [(128, 16, False), (128, 64, False), (128, 96, False), (128, 112, False),
                                            (64, 48, False), (256, 64, False), (256, 240, False), (128, 66, True),
                                            (256, 2, True)])
def test_append_rotates_a_part(D, rot, adjacent, fmt, dev):
    """Heads of which the first dims are rotated, by halves and in pairs."""
    from semi_ar_draft_round_amd import binding as B
    say(f"[blocks] rot {rot} of {D} fmt {fmt}")
    rng = np.random.default_rng(D + rot)
    Hq, Hkv, P, lens, n = 5, 3, 32, [29, 5000], 11
    rows = n * len(lens)
    xb, x = bf(rng.standard_normal((rows, Hq + 2 * Hkv, D)))
    wb, w = bf(1 + 0.4 * rng.standard_normal((2, D)))
    freq = 1e4 ** (-2.0 * np.arange(rot // 2) / rot)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)
    xt = t16(xb, dev)
    pages = (lens[1] + n) // P + 1
    table = torch.full((2, pages), -1, dtype=torch.int32, device=dev)
    for r, t in enumerate(lens):
        for i in range(t // P, (t + n - 1) // P + 1):
            table[r, i] = 4 * r + i - t // P
    pool = torch.zeros((8, B.dspark_cache_page_bytes(fmt, Hkv, D, P)), dtype=torch.uint8, device=dev)
    q = B.dspark_cache_append(xt[:, :Hq], xt[:, Hq:Hq + Hkv], xt[:, Hq + Hkv:], pool, table, i32(*lens), i32(n - 1, n - 1),
                              n - 1, fmt=fmt, page=P, wq=t16(wb[0], dev), wk=t16(wb[1], dev), eps=1e-5,
                              freq=torch.from_numpy(freq).to(dev), adjacent=adjacent)
    k, _ = B.dspark_cache_read(pool, table, i32(*lens), i32(n, n), n, fmt=fmt, page=P, heads_kv=Hkv, dim=D)
    pos = np.concatenate([t + np.arange(n) for t in lens])
    for name, got, heads, weight in ("q", back(q), slice(0, Hq), w[0]), ("k", back(k).reshape(rows, Hkv, D),
                                                                        slice(Hq, Hq + Hkv), w[1]):
        y = OC.norm(x[:, heads], weight, 1e-5)
        z = OC.rotate(y, pos, freq, adjacent)
        h = np.arange(rot // 2)
        a, b = (2 * h, 2 * h + 1) if adjacent else (h, h + rot // 2)
        mag = np.abs(y)
        mag[..., a] = mag[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
        if fmt == FP4 and name == "k":
            # half of the widest step is one unit 2^e, and top > 3.5 * 2^e
            top = np.abs(z).reshape(rows, Hkv, -1, 32).max(-1).repeat(32, -1)
            assert np.all(np.abs(got - z) <= top * (2 / 7) * (1 + 2.0 ** -20))
        else:
            assert np.all(np.abs(got - z) <= HALF * np.abs(z) + 64 * F32 * mag)
