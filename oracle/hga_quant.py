"""Float64 oracle of the 8-bit K/V cache (append, attention, eviction by accumulated weight).

One (sequence, KV head) at a time, in plain numpy, sharing no code with the CUDA path.  Groups of
16 tokens hold 8-bit codes and one float32 scale per tensor; the open group's rows stay unrounded.
The two quotients and the product of the code's definition are float32's, as the definition has
them; everything else is float64.
"""

from __future__ import annotations

import math

import numpy as np

GROUP = 16
PEAK = {"e4m3": 448.0, "int8": 127.0}


def code_values(fmt: str) -> np.ndarray:
    """The value of each of the 256 codes."""
    c = np.arange(256)
    if fmt == "int8":
        return np.where(c < 128, c, c - 256).astype(np.float64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def quantise(x: np.ndarray, fmt: str) -> tuple[np.ndarray, np.float32]:
    """(values of the codes, scale) of one group x [16, D] of float32 (or narrower) values."""
    x = np.asarray(x, dtype=np.float32)
    if not np.isfinite(x).all():
        return np.zeros(x.shape), np.float32(np.nan)
    amax = np.abs(x).max()
    if amax < 2.0 ** -100:
        return np.zeros(x.shape), np.float32(0)
    peak = np.float32(PEAK[fmt])
    scale, inverse = amax / peak, peak / amax      # float32 divisions
    y = (x * inverse).astype(np.float32).astype(np.float64)
    if fmt == "int8":
        return np.rint(y), scale
    # the nearest of the format's values, ties to the even mantissa
    e = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -30)))
    step = 2.0 ** (np.maximum(e, -6.0) - 3.0)
    return np.rint(y / step) * step, scale


class Item:
    """The cache of one (sequence, KV head)."""

    def __init__(self, fmt: str, dim: int):
        self.fmt, self.dim = fmt, dim
        self.k, self.v = [], []                    # live groups: (code values, scale)
        self.k_tail = np.zeros((0, dim))
        self.v_tail = np.zeros((0, dim))

    def append(self, k: np.ndarray, v: np.ndarray) -> None:
        for name, rows in (("k", k), ("v", v)):
            tail = np.concatenate([getattr(self, name + "_tail"), rows])
            while len(tail) >= GROUP:
                getattr(self, name).append(quantise(tail[:GROUP], self.fmt))
                tail = tail[GROUP:]
            setattr(self, name + "_tail", tail)

    def rows(self, name: str, entries) -> np.ndarray:
        got = [c * np.float64(s) for c, s in (getattr(self, name)[e] for e in entries)]
        return np.concatenate(got + [getattr(self, name + "_tail")]) if got else \
            getattr(self, name + "_tail")

    def attend(self, q: np.ndarray, entries=None):
        """(out [G, D], lse [G], weight of each table entry, open group last) of queries q [G, D]
        over the groups `entries` (all of them by default) and the tail."""
        entries = list(range(len(self.k))) if entries is None else list(entries)
        n_units = len(self.k) + (len(self.k_tail) > 0)
        weight = np.zeros(n_units)
        k, v = self.rows("k", entries), self.rows("v", entries)
        if not len(k):
            return np.zeros(q.shape), np.full(len(q), -np.inf), weight
        # a tail that holds an infinity or NaN stands as the group that it will be
        if not (np.isfinite(self.k_tail).all() and np.isfinite(self.v_tail).all()):
            return np.full(q.shape, np.nan), np.full(len(q), np.nan), np.full(n_units, np.nan)
        with np.errstate(invalid="ignore"):        # a group that holds a NaN makes NaN
            s = q @ k.T / math.sqrt(self.dim)
            top = s.max(1, keepdims=True)
            e = np.exp(s - top)
            lse = top[:, 0] + np.log(e.sum(1))
            p = e / e.sum(1, keepdims=True)
            out = p @ v
        for i, g in enumerate(entries):
            weight[g] = p[:, i * GROUP:(i + 1) * GROUP].sum()
        if len(self.k_tail):
            weight[-1] = p[:, len(entries) * GROUP:].sum()
        return out, lse, weight


def keep_groups(weight, n: int, keep: int, sink: int, recent: int) -> list[int]:
    """The groups of n that stay under a budget: the first `sink`, the last `recent`, and the
    heaviest of the rest (equal weights: the earlier; NaN least)."""
    if n <= keep:
        return list(range(n))
    middle = list(range(sink, n - recent))
    worth = {g: (-np.inf if np.isnan(weight[g]) else float(weight[g])) for g in middle}
    best = sorted(middle, key=lambda g: (np.isnan(weight[g]), -worth[g], g))[:keep - sink - recent]
    return list(range(sink)) + sorted(best) + list(range(n - recent, n))
