"""The attention's weights are not rounded to the pages' precision: its output
is as near to float64 as one rounding to bf16 allows.

Bound of the error: the output's own rounding, half a step of bf16 = 2^-8 of
it; and of sum_j p_j |v_j|: 2^-15 for a weight's two bf16 numbers (the upper
half of its bits leaves up to 2^-7 of it, of which the second number, the
nearest, loses 2^-8) and the 2^-22 that the second holds on top; 2^-24 for each
of 2 N + 64 additions and products of fp32, N tokens; and twice the score's
error, D + 8 roundings of 2^-24 of the sum of magnitudes |q| |k|."""

import numpy as np
import pytest

from cache_cases import BF16, F32, FP4, HALF
from oracle import cache as OC
from test_gpu_cache_attention import Case, back, dev, say  # noqa: F401  (dev: a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SHAPES = [  # lens, ells, Hq, Hkv, P, gamma, window, sinks
    ([0, 0], [0, 0], 8, 1, 64, 0, 0, 0),            # one visible token
    ([1, 2, 5], [0, 0, 0], 14, 2, 64, 0, 2, 0),     # two
    ([399, 7], [12, 3], 2, 2, 128, 12, 38, 0),
    ([700, 129], [16, 3], 14, 2, 64, 16, 0, 0),
    ([333, 40], [16, 2], 8, 2, 16, 16, 100, 4),
    ([2500], [0], 8, 8, 32, 0, 0, 0),
]


@pytest.mark.parametrize("fmt", [BF16, FP4])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(x) for x in s))
def test_as_near_as_one_rounding(shape, D, fmt, dev):
    lens, ells, Hq, Hkv, P, gamma, window, sinks = shape
    say(f"[weights] fmt {fmt} D {D} {shape}")
    c = Case(dev, fmt, lens, ells, Hq, Hkv, D, P, gamma, window, sinks, seed=D)
    out, _ = c.call(torch.zeros((c.rows, Hq, D), dtype=torch.bfloat16, device=dev))
    o = back(out)
    off = on = 0.0
    for r, (f, n) in enumerate(zip(c.first, c.n)):
        q, k, v, pos = c.nq[f:f + n], c.ks[r], c.vs[r], lens[r] + np.arange(n)
        want, _ = OC.attention(q, k, v, pos, c.scale, window, sinks)
        A, _ = OC.attention(q, k, np.abs(v), pos, c.scale, window, sinks)
        mag = (np.abs(q) * np.repeat(np.abs(k).max(axis=0), Hq // Hkv, axis=0)[None]).sum(-1) * c.scale
        share = 2.0 ** -15 + 2.0 ** -22 + (2 * k.shape[0] + 64) * F32 + 2 * (D + 8) * F32 * mag
        err = np.abs(o[f:f + n] - want)
        tol = HALF * np.abs(want) * (1 + HALF) + share[..., None] * A
        assert np.all(err <= tol), (r, float((err / tol).max()))
        off += (err ** 2).sum()
        on += (want ** 2).sum()
    say(f"  off {np.sqrt(off / on):.2e} of the output")
