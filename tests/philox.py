"""Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011) in numpy,
and the mask that dropout takes from it."""
import numpy as np

LOW = np.uint64(0xFFFFFFFF)


def philox4x32(counter, key, rounds=10):
    """counter: four uint64 arrays below 2^32; key: two integers.  Returns four arrays below 2^32."""
    c = [np.asarray(x, dtype=np.uint64) for x in counter]
    k = [int(key[0]), int(key[1])]
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & LOW, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]),
             a & LOW]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def keep_mask(n, p, seed, offset, first=0):
    """(mask of the n elements from `first` on, a multiple of 8, the factor of the kept ones)."""
    vec = np.arange(-(-n // 8), dtype=np.uint64) + np.uint64(first // 8)
    c = philox4x32([vec & LOW, vec >> np.uint64(32), np.full_like(vec, offset & 0xFFFFFFFF),
                    np.full_like(vec, offset >> 32)], (seed & 0xFFFFFFFF, seed >> 32))
    bits = np.empty((vec.size, 8), dtype=np.uint64)
    for i, w in enumerate(c):
        bits[:, 2 * i], bits[:, 2 * i + 1] = w & np.uint64(0xFFFF), w >> np.uint64(16)
    t = round(p * 65536)
    return bits.reshape(-1)[:n] >= t, (65536 / (65536 - t) if t < 65536 else 0.0)
