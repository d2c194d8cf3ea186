"""Float64 reference of the conditions on logits (include/dspark_logits.h)."""

from __future__ import annotations

import numpy as np


class History:
    """Which tokens a request's prompt holds and how often each was answered."""

    def __init__(self, V):
        self.V = V
        self.prompt = np.zeros(V, bool)
        self.count = np.zeros(V, np.int64)

    def start(self, tokens):
        self.prompt[:] = False
        self.count[:] = 0
        for t in tokens:
            if 0 <= t < self.V:
                self.prompt[t] = True

    def add(self, tokens):
        for t in tokens:
            if 0 <= t < self.V:
                self.count[t] = min(self.count[t] + 1, 32767)

    def words(self):
        return (self.count | np.where(self.prompt, 0x8000, 0)).astype(np.uint16)


def row(x, history, follows, repetition, presence, frequency, biases, allowed):
    """One row's logits x [V] (float64): `follows` the tokens of the round that
    come before it (not yet in the history); biases [(token, value)]; allowed
    [V] bool or None; history None: no penalties."""
    V = len(x)
    y = np.array(x, np.float64)
    if history is not None:
        n = history.count.copy()
        for t in follows:
            if 0 <= t < V:
                n[t] += 1
        seen = history.prompt | (n > 0)
        with np.errstate(invalid="ignore"):
            y = np.where(seen, np.where(y > 0, y / repetition, y * repetition), y)
            y = y - np.where(n > 0, frequency * n + presence, 0.0)
    for t, b in biases:
        if 0 <= t < V:
            y[t] += b
    if allowed is not None:
        y[~allowed] = -np.inf
    return y
