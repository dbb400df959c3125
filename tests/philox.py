"""Philox4x32-10 in numpy, from its definition (J. Salmon, M. Moraes, R. Dror,
D. Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011), and the mask that
dropout makes of it."""
import numpy as np


def philox(counter, key, rounds=10):
    """counter: four arrays or numbers of 32 bits; key: two numbers.  Four arrays of 32-bit words as uint64."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(key[0]), int(key[1])]
    for _ in range(rounds):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        low = np.uint64(0xFFFFFFFF)
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), q & low, (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return c


def words(m, n, seed, offset, first_row=0):
    """The word of every element of m x n."""
    at = offset % 2 ** 64
    groups = np.arange((n + 3) // 4, dtype=np.uint64)[None, :] + np.zeros((m, 1), dtype=np.uint64)
    rows = (np.arange(m, dtype=np.uint64) + np.uint64(first_row))[:, None] + np.zeros_like(groups)
    full = lambda v: np.full(groups.shape, v, dtype=np.uint64)  # noqa: E731
    w = philox((groups, rows, full(at % 2 ** 32), full(at >> 32)), (seed % 2 ** 32, seed >> 32))
    return np.stack(w, 2).reshape(m, -1)[:, :n]


def border(p):
    """Words below it drop their elements (p 2^32, ties to even: exact in 64 bits)."""
    return int(np.rint(np.float64(p) * 2.0 ** 32))
