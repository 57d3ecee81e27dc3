"""NumPy oracle of the dropout and its generator: TEST INFRASTRUCTURE ONLY (see
``oracle/__init__.py``); it shares no code with the HIP path.

Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as
1, 2, 3", SC 2011): ten rounds of two 32 x 32 bit products on a counter of four
words under a key of two, the key raised by two constants each round. Element
e of an array has 16 bits of the block at counter (e / 8, step, call).
"""

from __future__ import annotations

import numpy as np

__all__ = ["philox4x32", "dropout_bits", "dropout_threshold", "dropout"]


def philox4x32(counter, key, rounds=10):
    """Words [.., 4] of counters [.., 4] under the key (two words)."""
    c = [np.asarray(counter)[..., i].astype(np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(rounds):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & low,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return np.stack(c, -1).astype(np.uint32)


def dropout_bits(first, n, seed, step, call):
    """16 bits each of elements first .. first + n - 1."""
    e = np.arange(first, first + n, dtype=np.uint64)
    block = e // np.uint64(8)
    counter = np.stack([block & np.uint64(0xFFFFFFFF), block >> np.uint64(32),
                        np.full(n, step % 2 ** 32, np.uint64), np.full(n, call, np.uint64)], -1)
    words = philox4x32(counter, (seed % 2 ** 32, seed // 2 ** 32 % 2 ** 32))
    at = (e % np.uint64(8)).astype(np.int64)
    return (words[np.arange(n), at // 2] >> (16 * (at % 2)).astype(np.uint32)) & 0xFFFF


def dropout_threshold(p):
    return int(np.floor(p * 65536 + 0.5))


def dropout(x, p, seed, step, call, first=0):
    """x (flat, float32) with what is dropped at 0 and the rest scaled, rounded
    to float32 once; x holds the elements from ``first`` on."""
    x = np.asarray(x, np.float32)
    t = dropout_threshold(p)
    keep = dropout_bits(first, x.size, seed, step, call).reshape(x.shape) >= t
    if t == 65536:
        return np.zeros_like(x)
    with np.errstate(over="ignore", invalid="ignore"):
        return np.where(keep, x * np.float32(65536 / (65536 - t)), np.float32(0))
