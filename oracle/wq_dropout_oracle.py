"""Plain NumPy form of the counter-based dropout (test infrastructure).

Philox4x32-10 as its authors publish it (Salmon, Moraes, Dror, Shaw,
"Parallel random numbers: as easy as 1, 2, 3", 2011), word by word in 64-bit
integers, and the elements that it keeps.
"""

import numpy as np

_LOW = np.uint64(0xFFFFFFFF)


def philox4x32(counters, key, rounds=10):
    """uint32 [n][4] output words of the counters uint32 [n][4] under the key
    (k0, k1)."""
    c = [np.asarray(counters, dtype=np.uint64)[:, i] for i in range(4)]
    k0, k1 = (int(k) for k in key)
    for _ in range(rounds):
        p0 = c[0] * np.uint64(0xD2511F53)
        p1 = c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), p1 & _LOW,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p0 & _LOW]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, axis=1).astype(np.uint32)


def drop_halves(first, count, seed, offset):
    """uint16 draws of the elements first .. first + count - 1 (first a
    multiple of 8): eight to a block, low half of each word first."""
    groups = np.arange(first // 8, (first + count + 7) // 8, dtype=np.uint64)
    c = np.empty((groups.size, 4), dtype=np.uint32)
    c[:, 0], c[:, 1] = groups & _LOW, groups >> np.uint64(32)
    c[:, 2], c[:, 3] = offset & 0xFFFFFFFF, (offset >> 32) & 0xFFFFFFFF
    w = philox4x32(c, (seed & 0xFFFFFFFF, seed >> 32))
    return np.stack([w & 0xFFFF, w >> 16], axis=2).astype(np.uint16).reshape(-1)[:count]


def drop_keep(shape, p, seed, offset):
    """(kept [shape] bool, factor of the kept elements as float64)."""
    t = int(np.floor(p * 65536 + 0.5))
    n = int(np.prod(shape))
    return (drop_halves(0, n, seed, offset) >= t).reshape(shape), 65536 / (65536 - t)
