"""Helpers of the paged-cache tests: bf16 bits, page building, tolerances."""

import numpy as np

from oracle import cache as OC
from semi_ar_draft_round_amd.workloads import bf16_bits, bf16_to_f32

BF16, FP4 = 1, 2
HALF = 2.0 ** -8     # bf16: half a step relative to the value
F32 = 2.0 ** -24


def bf(x):
    """float -> (bits uint16, the float64 value they stand for)."""
    b = bf16_bits(np.asarray(x, dtype=np.float32))
    return b, bf16_to_f32(b).astype(np.float64)


def make_tokens(rng, fmt, T, H, D, spread=1.0):
    """What a cache of T tokens holds: stored K and V for write_pages and the
    float64 values they stand for."""
    if fmt == BF16:
        kb, k = bf(rng.standard_normal((T, H, D)) * spread)
        vb, v = bf(rng.standard_normal((T, H, D)))
        return kb, vb, k, v
    E = D // 32
    kc = rng.integers(0, 16, (T, H, D)).astype(np.uint8)
    kb = rng.integers(123, 127, (T, H, E)).astype(np.uint8)
    vc = rng.integers(0, 16, (T, H, D)).astype(np.uint8)
    vs = rng.uniform(0.1, 0.6, (T, H)).astype(np.float32)
    sign = lambda c: np.where(c & 8, -1.0, 1.0) * OC.E2M1[c & 7]
    k = sign(kc) * np.repeat(np.exp2(kb.astype(np.float64) - 127) * spread, 32, axis=-1)
    kb = (kb.astype(np.int64) + int(np.log2(spread))).astype(np.uint8)
    return (kc, kb), (vc, vs), k, sign(vc) * vs.astype(np.float64)[..., None]


def page_bytes(fmt, H, D, P):
    return H * P * (4 * D if fmt == BF16 else D + D // 32 + 4)


def attention_tolerance(q, k, v, pos, scale, window, sinks, o, have=None):
    """Bounds of the kernel's error in out and lse, from its roundings.

    A score is an fp32 sum of D exact products and a few scalings: off by at
    most (D + 8) 2^-24 of the sum of magnitudes, and its exponential by as
    much again in relative terms (e^x - 1 < 2 x).  A weight is rounded to
    bf16 (half a step, 2^-8), as for 4 bits its product with the V scale.
    The sums over N tokens are fp32, in any order: N + 64 roundings of
    2^-24.  The result is rounded to bf16 once."""
    D, N = q.shape[2], k.shape[0]
    finite = np.nan_to_num(np.abs(v), nan=0.0, posinf=0.0)
    A, _ = OC.attention(q, k, finite, pos, scale, window, sinks, have)
    G = q.shape[1] // k.shape[1]
    ka = np.nan_to_num(np.abs(k), nan=0.0, posinf=0.0).max(axis=0)          # [Hkv][D]
    mag = (np.abs(q) * np.repeat(ka, G, axis=0)[None]).sum(-1) * abs(scale)  # [rows][Hq]
    delta = 2 * (D + 8) * F32 * mag
    n = (N + 64) * F32
    return HALF * np.abs(o) + (HALF * (1 + HALF) + delta + n)[..., None] * A + 1e-30, delta + n + 1e-6


def build(rng, fmt, lens, H, D, P, max_pages, spare=3, garbage=0xFF):
    """A pool whose unwritten bytes are all `garbage` (0xFF: NaNs), a shuffled
    table, and every request's dense values.  Returns pool, table, [k], [v]."""
    need = [-(-n // P) for n in lens]
    N = sum(need) + spare
    ids = rng.permutation(N)
    table = np.full((len(lens), max_pages), -1, dtype=np.int32)
    pool = np.full((N, page_bytes(fmt, H, D, P)), garbage, dtype=np.uint8)
    at, ks, vs = 0, [], []
    for r, (n, m) in enumerate(zip(lens, need)):
        table[r, :m] = ids[at:at + m]
        at += m
        sk, sv, k, v = make_tokens(rng, fmt, n, H, D)
        if n:
            OC.write_pages(fmt, sk, sv, table[r], P, pool)
        ks.append(k)
        vs.append(v)
    return pool, table, ks, vs
