"""Dropout from a counter-based generator: a plain statement of what the library's
monarch_dropout computes, with Philox4x32-10 over Python integers held in numpy's
64-bit words. TEST INFRASTRUCTURE ONLY (it shares no code with the HIP path)."""
from __future__ import annotations

import numpy as np

M32 = np.uint64(0xFFFFFFFF)
S32 = np.uint64(32)


def philox(counter, key):
    """Philox4x32-10: counter [n, 4] and key (2 words) to [n, 4] words."""
    c = [np.asarray(counter[:, i], dtype=np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)   # below 2^64
        c = [(b >> S32) ^ c[1] ^ np.uint64(k[0]), b & M32, (a >> S32) ^ c[3] ^ np.uint64(k[1]), a & M32]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, axis=1)


def draws(n, seed, offset, first=0):
    """16 bits for each of the elements [first, first + n)."""
    unit = np.arange(first // 8, (first + n + 7) // 8, dtype=np.uint64)
    ctr = np.stack([unit & M32, unit >> S32, np.full_like(unit, offset & 0xFFFFFFFF), np.full_like(unit, offset >> 32)], axis=1)
    w = philox(ctr, (seed & 0xFFFFFFFF, seed >> 32))
    halves = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], axis=2).reshape(-1)
    at = first % 8
    return halves[at:at + n].astype(np.int64)


def dropout(x, p, seed, offset, residual=None):
    """y in 64 bits, and which elements are kept."""
    t = int(np.floor(p * 65536 + 0.5))
    keep = (draws(x.size, seed, offset) >= t).reshape(x.shape)
    y = np.where(keep, x.astype(np.float64) * (65536.0 / (65536 - t) if t < 65536 else 0.0), 0.0)
    return (y if residual is None else residual.astype(np.float64) + y), keep
