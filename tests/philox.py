"""Philox4x32-10 in numpy, from the paper (Salmon et al., Parallel random numbers: as easy as 1, 2, 3, SC 2011)."""
import numpy as np

M = (np.uint64(0xD2511F53), np.uint64(0xCD9E8D57))
W = (0x9E3779B9, 0xBB67AE85)
LOW, HALF = np.uint64(0xFFFFFFFF), np.uint64(32)


def philox(counter, key):
    """counter: four arrays (or numbers) of 32-bit words, key: two; returns four arrays of words."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(v) for v in key]
    for _ in range(10):
        a, b = c[0] * M[0], c[2] * M[1]
        c = [(b >> HALF) ^ c[1] ^ np.uint64(k[0]), b & LOW, (a >> HALF) ^ c[3] ^ np.uint64(k[1]), a & LOW]
        k = [(k[0] + W[0]) & 0xFFFFFFFF, (k[1] + W[1]) & 0xFFFFFFFF]
    return c


def keep_mask(rows, F, p, seed, offset):
    """The elements that dropout with probability p keeps."""
    seed, offset = seed & (2 ** 64 - 1), offset & (2 ** 64 - 1)
    blocks = (F + 3) // 4
    c0 = np.broadcast_to(np.arange(blocks), (rows, blocks))
    c1 = np.broadcast_to(np.arange(rows)[:, None], (rows, blocks))
    w = philox((c0, c1, offset & 0xFFFFFFFF, offset >> 32), (seed & 0xFFFFFFFF, seed >> 32))
    words = np.stack([np.broadcast_to(v, (rows, blocks)) for v in w], -1).reshape(rows, 4 * blocks)[:, :F]
    return words >= np.uint64(int(p * 2 ** 32))
