"""The dropout's generator, Philox 4 x 32 with ten rounds (Salmon, Moraes, Dror and Shaw,
"Parallel random numbers: as easy as 1, 2, 3", 2011), and the mask made of its words, in
numpy integers of 64 bits.  Test code only."""
import numpy as np

M32 = np.uint64(0xffffffff)


def philox(counter, key):
    """counter [..., 4], key (k0, k1): the words [..., 4], all 32-bit values."""
    c = [np.asarray(counter)[..., i].astype(np.uint64) for i in range(4)]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(10):
        p, q = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), q & M32,
             (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p & M32]
        k0, k1 = (k0 + 0x9E3779B9) & 0xffffffff, (k1 + 0xBB67AE85) & 0xffffffff
    return np.stack(c, -1)


def keep_mask(rows, width, p, seed, offset, site=0):
    """(mask [len(rows), width], the factor of what is kept) for row numbers ``rows``."""
    blocks = (width + 3) // 4
    at = np.asarray(rows, dtype=np.uint64)[:, None] * np.uint64(blocks) + np.arange(blocks, dtype=np.uint64)
    seed, offset = int(seed) % 2 ** 64, int(offset) % 2 ** 64
    c = np.empty(at.shape + (4,), dtype=np.uint64)
    c[..., 0] = at & M32
    c[..., 1] = (at >> np.uint64(32)) | np.uint64(site << 16)
    c[..., 2], c[..., 3] = offset & 0xffffffff, offset >> 32
    words = philox(c, (seed & 0xffffffff, seed >> 32)).reshape(len(at), 4 * blocks)[:, :width]
    limit = round(p * 2.0 ** 32)
    return words >= np.uint64(limit), 1.0 / (1.0 - limit / 2.0 ** 32)
