"""fp64 NumPy oracle of the 4-bit K/V cache operators (test infrastructure).

Written from the definitions in ``include/ulysses.h`` with none of the
library's code: rows are handled one group at a time, codes one nibble at a
time.  Cache bytes are split and joined here too, so a test can compare a
cache bit for bit.
"""
from __future__ import annotations

import numpy as np

BLOCK, BLOCK_BYTES, D = 32, 4608, 128


def bf16_to_f64(bits: np.ndarray) -> np.ndarray:
    """float64 values of bf16 bit patterns (uint16)."""
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f64_to_bf16(x: np.ndarray) -> np.ndarray:
    """Nearest bf16 bit patterns, ties to even (NaN -> 0x7fc0); x must be exact or rounded to
    float64 only, so there is one rounding."""
    x = np.asarray(x, dtype=np.float64)
    out = np.empty(x.shape, dtype=np.uint16)
    flat, res = x.ravel(), out.ravel()
    for i, v in enumerate(flat):
        if np.isnan(v):
            res[i] = 0x7FC0
            continue
        sign = 0x8000 if np.signbit(v) else 0
        a = abs(v)
        if a == 0:
            res[i] = sign
            continue
        if np.isinf(a):
            res[i] = sign | 0x7F80
            continue
        e = max(int(np.floor(np.log2(a))), -126)
        while a >= 2.0 ** (e + 1):
            e += 1
        while e > -126 and a < 2.0 ** e:
            e -= 1
        n = np.rint(a / 2.0 ** (e - 7))          # 128..256 for normal numbers
        v = n * 2.0 ** (e - 7)
        if v >= 2.0 ** 128:
            res[i] = sign | 0x7F80
        else:
            res[i] = sign | int(np.float32(v).view(np.uint32) >> 16)
    return out.reshape(x.shape)


def quantise_group(x: np.ndarray):
    """Codes [64] and the (s, m) bit patterns of 64 bf16 values given in float64."""
    bad = (np.zeros(64, dtype=np.uint8), 0x7FC0, 0x7FC0)
    if not np.all(np.isfinite(x)):
        return bad
    m = float(x.min())
    spread = np.float64(x.max()) - m
    if spread > 3.4028235677973366e38:           # not a finite fp32 difference
        return bad
    sb = int(f64_to_bf16(np.array([spread / 15]))[0])
    s = float(bf16_to_f64(np.array([sb], dtype=np.uint16))[0])
    codes = np.zeros(64, dtype=np.uint8)
    if s > 0:
        codes = np.clip(np.rint((x - m) / s), 0, 15).astype(np.uint8)
    return codes, sb, int(f64_to_bf16(np.array([m]))[0])


def quantise_row(x: np.ndarray):
    """The 64 code bytes and the four uint16 (s0, m0, s1, m1) of a row of 128."""
    codes = np.zeros(128, dtype=np.uint8)
    meta = np.zeros(4, dtype=np.uint16)
    for w in (0, 1):
        codes[64 * w:64 * w + 64], meta[2 * w], meta[2 * w + 1] = quantise_group(x[64 * w:64 * w + 64])
    rows = np.zeros(64, dtype=np.uint8)
    for d in range(0, 128, 2):
        w, r = divmod(d, 64)
        g, i = divmod(r, 8)
        rows[8 * g + 4 * w + i // 2] = codes[d] | (codes[d + 1] << 4)
    return rows, meta


class Cache:
    """The three arrays of a cache's bytes, as writable views."""

    def __init__(self, raw: np.ndarray, batch: int, heads: int, capacity: int):
        n = batch * heads * capacity
        nb = n // BLOCK * BLOCK_BYTES
        assert raw.dtype == np.uint8 and raw.size == nb + 8 * n
        self.blocks = raw[:nb].reshape(batch, heads, capacity // BLOCK, BLOCK_BYTES)
        self.weight = raw[nb:nb + 4 * n].view(np.float32).reshape(batch, heads, capacity)
        self.pos = raw[nb + 4 * n:].view(np.int32).reshape(batch, heads, capacity)

    def row(self, b: int, h: int, slot: int, plane: int) -> np.ndarray:
        """The 64 code bytes of a slot (plane 0: K, 1: V)."""
        return self.blocks[b, h, slot // BLOCK, 2048 * plane + 64 * (slot % BLOCK):][:64]

    def meta(self, b: int, h: int, slot: int, plane: int) -> np.ndarray:
        at = 4096 + 16 * (slot % BLOCK) + 8 * plane
        return self.blocks[b, h, slot // BLOCK, at:at + 8].view(np.uint16)

    def values(self, b: int, h: int, lo: int, hi: int, plane: int):
        """float64 rows [hi - lo, 128] of slots lo..hi, with their steps s [hi - lo, 2]."""
        n = max(hi - lo, 0)
        raw = np.zeros((n, 64), dtype=np.int64)
        sm = np.zeros((n, 4))
        for j, slot in enumerate(range(lo, hi)):
            raw[j] = self.row(b, h, slot, plane)
            sm[j] = bf16_to_f64(self.meta(b, h, slot, plane))
        codes = np.zeros((n, D))
        for g in range(8):
            for w in range(2):
                for i in range(4):
                    byte = raw[:, 8 * g + 4 * w + i]
                    codes[:, 64 * w + 8 * g + 2 * i] = byte % 16
                    codes[:, 64 * w + 8 * g + 2 * i + 1] = byte // 16
        out = np.zeros((n, D))
        for w in (0, 1):
            out[:, 64 * w:64 * w + 64] = sm[:, 2 * w + 1:2 * w + 2] + sm[:, 2 * w:2 * w + 1] * codes[:, 64 * w:64 * w + 64]
        return out, sm[:, 0::2]


def kept_slots(weight: np.ndarray, n: int, keep: int, sink: int, recent: int) -> np.ndarray:
    """The slots of one pair that an eviction keeps, ascending."""
    if n <= keep:
        return np.arange(n)
    free = list(range(sink, n - recent))
    rank = {t: (-np.inf if np.isnan(weight[t]) else float(weight[t]), not np.isnan(weight[t])) for t in free}
    free.sort(key=lambda t: (-rank[t][0], not rank[t][1], t))
    chosen = list(range(sink)) + list(range(n - recent, n)) + free[:keep - sink - recent]
    return np.array(sorted(chosen))


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float):
    """Softmax attention of one query row over rows k, v: (o, base-2 log-sum, p)."""
    if k.shape[0] == 0:
        return np.zeros(D), -np.inf, np.zeros(0)
    z = scale * (k @ q)
    top = z.max()
    e = np.exp(z - top)
    total = e.sum()
    return (e / total) @ v, (top + np.log(total)) / np.log(2.0), e / total
