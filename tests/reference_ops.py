"""Plain 64-bit implementations the operator tests compare with, written from the definitions in
``include/hwkv.h``: 8-bit groups and rings of them, and attention over a ring with capped or
distance-biased scores.  numpy only, no code of the package."""
from __future__ import annotations

import math

import numpy as np

GROUP = 16
MIN_EXP = -120


def nearest_e4m3(y: np.ndarray) -> np.ndarray:
    """The e4m3 value nearest to y, |y| <= 448, ties to even: the numbers are multiples of 2^-9
    below 2^-6 and of 2^(x - 3) in [2^x, 2^(x + 1)) above."""
    _, x = np.frexp(np.abs(y))              # |y| = f * 2^x, f in [1/2, 1)
    step = np.ldexp(1.0, np.maximum(x - 1, -6) - 3)
    return np.rint(y / step) * step         # rint rounds halves to even


def encode_group(x: np.ndarray):
    """Codes (as values) and scale of one group of rows [16, D]."""
    fine = np.isfinite(x)
    amax = float(np.abs(np.where(fine, x, 0.0)).max())
    e = MIN_EXP
    while 448.0 * 2.0 ** e < amax:
        e += 1
    codes = nearest_e4m3(np.where(fine, x, 0.0) / 2.0 ** e)
    return np.where(fine, codes, np.nan), 2.0 ** e


class Ring8:
    """One head's ring of an 8-bit pool: codes [2, C, D] (as values) and scales [2, C / 16]."""

    def __init__(self, window: int, block_size: int, head_dim: int):
        self.w, self.C = window, -(-window // block_size) * block_size
        self.codes = np.zeros((2, self.C, head_dim))
        self.scales = np.zeros((2, self.C // GROUP))

    def _position(self, slot: int, newest: int) -> int:
        """The position slot holds once `newest` is stored, or -1 when it is outside the window."""
        p = newest - (newest - slot) % self.C
        return p if p >= 0 and p > newest - self.w else -1

    def _store(self, kv: int, g: int, rows: np.ndarray):
        self.codes[kv, g * GROUP:(g + 1) * GROUP], self.scales[kv, g] = encode_group(rows)

    def materialize(self, k: np.ndarray, v: np.ndarray, length: int):
        for g in range(self.C // GROUP):
            pos = [self._position(g * GROUP + j, length - 1) for j in range(GROUP)]
            if length < 1 or max(pos) < 0:
                continue
            for kv, src in enumerate((k, v)):
                self._store(kv, g, np.stack([src[p] if p >= 0 else np.zeros(src.shape[-1]) for p in pos]))

    def append(self, k: np.ndarray, v: np.ndarray, pos: int):
        g = pos % self.C // GROUP
        for kv, new in enumerate((k, v)):
            rows = self.values(kv)[g * GROUP:(g + 1) * GROUP].copy()
            for j in range(GROUP):
                p = self._position(g * GROUP + j, pos)
                rows[j] = new if p == pos else (rows[j] if p >= 0 else 0.0)
            self._store(kv, g, rows)

    def values(self, kv: int) -> np.ndarray:
        scale = np.repeat(self.scales[kv], GROUP)[:, None]
        return np.where(scale == 0.0, 0.0, self.codes[kv] * scale)

    def resident(self, length: int):
        """(positions, K rows, V rows) of the window at this length."""
        p = np.arange(max(0, length - self.w), length)
        return p, self.values(0)[p % self.C], self.values(1)[p % self.C]


def attention(q, k, v, scale, distance, cap=0.0, slope=0.0):
    """q [D], k and v [n, D], distance [n]: (softmax(score) v, sum of softmax |v|, largest |score|)."""
    if len(k) == 0:
        return np.zeros(v.shape[-1]), np.zeros(v.shape[-1]), 0.0
    s = k @ q * scale
    if cap > 0:
        s = cap * np.tanh(s / cap)
    s = s - slope * distance
    p = np.exp(s - s.max())
    p /= p.sum()
    return p @ v, p @ np.abs(v), float(np.abs(s).max())


def rope_frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    """(radians per position of each pair, magnitude)."""
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "by_parts":
        out = []
        for x in f:
            keep = (original_len * x / (2 * math.pi) - beta_slow) / (beta_fast - beta_slow)
            keep = min(1.0, max(0.0, keep))
            out.append(x * keep + x / factor * (1.0 - keep))
        return out, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rope(x, pos, freqs, layout, magnitude=1.0):
    """x [..., D] at one position, rotated in its first 2 len(freqs) dims."""
    y = np.array(x, dtype=np.float64)
    half = len(freqs)
    for i, f in enumerate(freqs):
        a, b = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
        c, s = math.cos(pos * f) * magnitude, math.sin(pos * f) * magnitude
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y
