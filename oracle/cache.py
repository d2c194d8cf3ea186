"""Float64 reference of the paged cache (include/dspark_cache.h), plain
definitions on dense arrays: no pages inside the mathematics.

Tokens of a request are rows of dense [tokens][heads][dim] arrays here; the
page functions at the end follow the layouts and the ownership rules.
"""

from __future__ import annotations

import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
BF16, FP4 = 1, 2


def norm(x, w, eps):
    """x / sqrt(mean(x^2) + eps) * w over the last axis (w None: x)."""
    x = np.asarray(x, dtype=np.float64)
    return x if w is None else x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(w, np.float64)


def rotate(x, pos, freq, adjacent):
    """x [rows][heads][D], pos [rows]: pairs turned by pos * freq (freq None: x)."""
    if freq is None or len(freq) == 0:
        return x
    h = len(freq)
    a = np.arange(h) * 2 if adjacent else np.arange(h)
    b = a + 1 if adjacent else a + h
    t = np.asarray(pos, np.float64)[:, None, None] * np.asarray(freq, np.float64)
    y = x.copy()
    y[..., a] = x[..., a] * np.cos(t) - x[..., b] * np.sin(t)
    y[..., b] = x[..., b] * np.cos(t) + x[..., a] * np.sin(t)
    return y


def _nearest(y):
    """Index of the nearest E2M1 magnitude, ties to the even code."""
    far = np.abs(y[..., None] - E2M1)
    tie = far == far.min(axis=-1, keepdims=True)
    even = tie & (np.arange(8) % 2 == 0)
    return np.where(even.any(-1), even.argmax(-1), tie.argmax(-1))


def quantise_k(k):
    """k [..., D] -> the values its 4-bit codes stand for (a 2^e per 32 dims)."""
    g = np.asarray(k, np.float64).reshape(*k.shape[:-1], -1, 32)
    top = np.abs(g).max(-1, keepdims=True)
    bad = ~(top < 2.0 ** 128)
    e = np.where((top > 0) & ~bad, np.frexp(np.where(bad, 1, top))[1] - 1, -200) - 2
    e = np.where(np.where(bad, 1, top) * np.exp2(-e.astype(np.float64)) > 7, e + 1, e)
    step = np.exp2(np.clip(e, -126, 125).astype(np.float64))
    v = E2M1[_nearest(np.abs(np.where(bad, 0, g)) / step)] * step * np.sign(g)
    return np.where(bad, np.nan, v).reshape(k.shape)


def quantise_v(v):
    """v [..., D] -> the values its codes stand for (one fp32 scale max/6)."""
    v = np.asarray(v, np.float64)
    top = np.abs(v).max(-1, keepdims=True)
    bad = ~np.isfinite(top)
    t = np.where(bad | (top == 0), 1, top)
    unit = (t.astype(np.float32) / np.float32(6)).astype(np.float64)
    # the borders are exact multiples of max / 12 and the like: 6 |v| against code * max
    far = np.abs(6 * np.abs(np.where(bad, 0, v))[..., None] - E2M1 * t[..., None])
    tie = far == far.min(-1, keepdims=True)
    even = tie & (np.arange(8) % 2 == 0)
    idx = np.where(even.any(-1), even.argmax(-1), tie.argmax(-1))
    return np.where(bad, np.nan, E2M1[idx] * unit * np.sign(v))


def attention(q, k, v, pos, scale, window, sinks, have=None):
    """q [rows][Hq][D] at positions pos; k, v [tokens][Hkv][D]; have [tokens]:
    False where the token has no page.  Returns out, lse."""
    rows, Hq, D = q.shape
    Hkv = k.shape[1]
    j = np.arange(k.shape[0])
    out, lse = np.zeros((rows, Hq, D)), np.full((rows, Hq), -np.inf)
    for i in range(rows):
        see = j <= pos[i]
        if window:
            see &= (j > pos[i] - window) | (j < sinks)
        if have is not None:
            see &= have
        if not see.any():
            continue
        ks, vs = k[see].astype(np.float64), v[see].astype(np.float64)
        for h in range(Hq):
            s = ks[:, h // (Hq // Hkv)] @ q[i, h].astype(np.float64) * scale
            m = s.max()
            p = np.exp(s - m)
            out[i, h] = p @ vs[:, h // (Hq // Hkv)] / p.sum()
            lse[i, h] = m + np.log(p.sum())
    return out, lse


# ---------------------------------------------------------------- pages

def write_pages(fmt, k, v, table, P, pool):
    """Dense tokens of one request (what the cache stands for, exactly) into
    pages: bf16 bits [tokens][Hkv][D] (uint16), or for FP4 the tuple
    (codes_k, bytes_k, codes_v, scale_v).  pool uint8 [n_pages][bytes]."""
    codes_k, bytes_k, codes_v, scale_v = (k, None, v, None) if fmt == BF16 else (k[0], k[1], v[0], v[1])
    T, H, D = codes_k.shape
    hb = pool.shape[1] // H
    for t in range(T):
        page, i = pool[table[t // P]], t % P
        b, u = i // 16, i % 16
        for h in range(H):
            head = page[h * hb:(h + 1) * hb]
            if fmt == BF16:
                w = head.view(np.uint16)
                kb = w[b * 16 * D:(b + 1) * 16 * D].reshape(D // 8, 16, 8)
                kb[:, u] = codes_k[t, h].reshape(D // 8, 8)
                vb = w[P * D + b * 16 * D:P * D + (b + 1) * 16 * D].reshape(2, D, 8)
                vb[u // 8, :, u % 8] = codes_v[t, h]
                continue
            E = D // 32
            kb = head[b * 8 * D:(b + 1) * 8 * D].reshape(E, 16, 16)
            c = codes_k[t, h].reshape(E, 32)
            kb[:, u] = c[:, 0::2] | c[:, 1::2] << 4
            head[P * D // 2 + i * E:P * D // 2 + (i + 1) * E] = bytes_k[t, h]
            at = P * (D // 2 + E)
            vb = head[at + b * 8 * D:at + (b + 1) * 8 * D].reshape(2, 32, E, 4)
            c = codes_v[t, h].reshape(E, 32).T
            byte = vb[u // 8, :, :, u % 8 // 2]
            vb[u // 8, :, :, u % 8 // 2] = (byte & 0x0F | c << 4) if u % 2 else (byte & 0xF0 | c)
            head[P * (D + E):].view(np.float32)[i] = scale_v[t, h]


class Pages:
    """Who owns which page, one request at a time."""

    def __init__(self, R, n_pages, max_pages, P):
        self.R, self.N, self.M, self.P = R, n_pages, max_pages, P
        self.table = np.full((R, max_pages), -1, dtype=np.int64)
        self.len = np.zeros(R, dtype=np.int64)

    def refs(self):
        """Table entries that name each page."""
        ref = np.zeros(self.N, dtype=np.int64)
        for p in self.table.flatten():
            if p >= 0:
                ref[p] += 1
        return ref

    def reserve(self, ell, gamma):
        """Returns ell_out, pairs, refused."""
        P = self.P
        ref = self.refs()
        free = [p for p in range(self.N) if ref[p] == 0]
        old = self.table.copy()
        out, pairs, refused, short, asked = [], [], False, False, {}
        total = 0
        for r in range(self.R):
            n = min(max(int(ell[r]), -1), gamma) + 1
            L = int(self.len[r])
            last = -(-(L + n) // P)
            if n == 0 or last > self.M:
                out.append(-1)
                refused |= n > 0
                continue
            first = L // P
            need = [i for i in range(first, last) if old[r, i] < 0]
            tail = old[r, first] if L % P else -1
            shared = tail >= 0 and ref[tail] > 1
            copy = exempt = False
            if shared:
                copy = ref[tail] - asked.get(tail, 0) > 1
                exempt = not copy
                asked[tail] = asked.get(tail, 0) + 1
            cnt = len(need) + copy
            before, total = total, total + cnt
            if (cnt and total > len(free)) or (exempt and before > len(free)):
                out.append(-1)
                refused = True
                continue
            ids = free[before:total]
            if copy:
                pairs.append((int(tail), ids[0]))
                self.table[r, first] = ids.pop(0)
            for i, p in zip(need, ids):
                self.table[r, i] = p
            out.append(n - 1)
        return out, pairs, refused

    def commit(self, ell, n_acc, gamma, window, sinks):
        P = self.P
        for r in range(self.R):
            n = min(max(int(ell[r]), -1), gamma) + 1
            if n == 0:
                continue
            self.len[r] = min(self.M * P, self.len[r] + min(max(int(n_acc[r]), 0), n - 1) + 1)
            for i in range(self.M):
                past = i * P >= self.len[r]
                unseen = window > 0 and (i + 1) * P - 1 <= self.len[r] - window and i * P >= sinks
                if past or unseen:
                    self.table[r, i] = -1

    def fork(self, parent):
        table, length = self.table.copy(), self.len.copy()
        for r in range(self.R):
            s = int(parent[r])
            if s == r or s < -1 or s >= self.R:
                continue
            self.table[r] = -1
            self.len[r] = 0
            if s >= 0:
                n = -(-int(length[s]) // self.P)
                self.table[r, :n] = table[s, :n]
                self.len[r] = length[s]

    def compact(self):
        ref = self.refs()
        U = int((ref > 0).sum())
        src = [p for p in range(U, self.N) if ref[p] > 0]
        dst = [p for p in range(U) if ref[p] == 0]
        to = dict(zip(src, dst))
        self.table = np.vectorize(lambda p: to.get(p, p), otypes=[np.int64])(self.table)
        return list(zip(src, dst))
