"""Helpers of the 8-bit cache's tests: pages built from the oracle's blocks."""

import numpy as np

from oracle import cache as OC
from cache_cases import bf

FP8 = 4


def page_bytes8(H, D, P):
    return H * (2 * P * D + 16)


def make_rows(rng, T, H, D, spread=1.0, by=7):
    """T tokens of H heads, taken in `by` at a time as a cache grows: [Rows8] of
    K and of V."""
    ks, vs = [], []
    for out, s in ((ks, spread), (vs, 1.0)):
        for _ in range(H):
            x = bf(rng.standard_normal((T, D)) * s * np.exp(0.3 * rng.standard_normal((T, 1))))[1]
            rows = OC.Rows8(D)
            for a in range(0, T, by):
                rows.append(a, x[a:a + by])
            out.append(rows)
    return ks, vs


def dense(rows):
    """[Rows8] of every head -> float64 [tokens][heads][D]"""
    return np.stack([r.values() for r in rows], axis=1)


def build8(rng, lens, H, D, P, max_pages, spare=3, garbage=0xFF, spread=1.0):
    """As cache_cases.build, for 8-bit pages; also the oracle's rows."""
    need = [-(-n // P) for n in lens]
    N = sum(need) + spare
    ids = rng.permutation(N)
    table = np.full((len(lens), max_pages), -1, dtype=np.int32)
    pool = np.full((N, page_bytes8(H, D, P)), garbage, dtype=np.uint8)
    at, ks, vs, rows = 0, [], [], []
    for r, (n, m) in enumerate(zip(lens, need)):
        table[r, :m] = ids[at:at + m]
        at += m
        k, v = make_rows(rng, n, H, D, spread)
        if n:
            OC.write_pages8(k, v, table[r], P, pool)
        ks.append(dense(k) if n else np.zeros((0, H, D)))
        vs.append(dense(v) if n else np.zeros((0, H, D)))
        rows.append((k, v))
    return pool, table, ks, vs, rows
