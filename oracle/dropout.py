"""The residual add with dropout in float64 (numpy): test infrastructure.

Philox4x32-10 written from its paper (Salmon, Moraes, Dror and Shaw, "Parallel
random numbers: as easy as 1, 2, 3", 2011: Section 3.3 and its constants) on
64-bit words, and the norm's gradients from oracle.block."""
from __future__ import annotations

import numpy as np

from . import block

_LOW = np.uint64(0xFFFFFFFF)
_SHIFT = np.uint64(32)


def philox(counter, key, rounds=10):
    """counter [..., 4] and key [2] of 32-bit words -> [..., 4] words."""
    x = [np.asarray(counter[..., i], np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    for _ in range(rounds):
        p0, p1 = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(p1 >> _SHIFT) ^ x[1] ^ np.uint64(k[0]), p1 & _LOW,
             (p0 >> _SHIFT) ^ x[3] ^ np.uint64(k[1]), p0 & _LOW]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(x, -1)


def halves(v):
    v = int(v) & 0xFFFFFFFFFFFFFFFF
    return v & 0xFFFFFFFF, v >> 32


def kept(rows, cols, p, seed, offset):
    """The mask [rows, cols]."""
    quads = (cols + 3) // 4
    c = np.zeros((rows, quads, 4), np.uint64)
    c[..., 0] = np.arange(quads, dtype=np.uint64)[None, :]
    c[..., 1] = np.arange(rows, dtype=np.uint64)[:, None]
    c[..., 2], c[..., 3] = halves(offset)
    words = philox(c, halves(seed)).reshape(rows, 4 * quads)[:, :cols]
    return words >= np.uint64(min(round(p * 2.0 ** 32), 2 ** 32 - 1))


def add_norm(x, residual, weight, scale, p, keep, eps):
    r = np.where(keep, x * (scale / (1.0 - p)), 0.0) + (0.0 if residual is None else residual)
    return block.norm(r, weight, eps), r


def add_norm_backward(r, weight, dy, dro, scale, p, keep, eps):
    ref = block.add_norm_backward(r, weight, dy, dro, 1.0, eps)
    ref["dx"] = np.where(keep, ref["dresidual"] * (scale / (1.0 - p)), 0.0)
    return ref
