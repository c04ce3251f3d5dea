"""The dropout mask of include/dropout.h on the host, word by word (numpy)."""
import numpy as np

M32 = 0xFFFFFFFF


def philox(counter, key):
    """Philox4x32-10: four 32-bit words (as uint64 arrays) from four counter words and two
    key words."""
    low, shift = np.uint64(M32), np.uint64(32)
    x = [np.asarray(c, dtype=np.uint64) for c in counter]
    for i in range(10):
        k0, k1 = (np.uint64((key[j] + i * step) & M32) for j, step in ((0, 0x9E3779B9), (1, 0xBB67AE85)))
        p, q = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(q >> shift) ^ x[1] ^ k0, q & low, (p >> shift) ^ x[3] ^ k1, p & low]
    return x


def threshold(drop):
    return int(np.rint(np.float64(np.float32(drop)) * 65536))


def scale(drop):
    t = threshold(drop)
    return 0.0 if t == 65536 else float(np.float32(65536 / (65536 - t)))


def keeps(m, n, drop, seed, offset):
    """Boolean [m, n]: which elements stay."""
    groups = -(-n // 8)
    offset %= 1 << 64
    words = philox([np.broadcast_to(np.arange(groups, dtype=np.uint64), (m, groups)),
                    np.broadcast_to(np.arange(m, dtype=np.uint64)[:, None], (m, groups)),
                    offset & M32, offset >> 32], [seed & M32, seed >> 32])
    bits = np.empty((m, groups, 8), dtype=np.uint16)
    for i, w in enumerate(words):
        bits[:, :, 2 * i], bits[:, :, 2 * i + 1] = w & np.uint64(0xFFFF), w >> np.uint64(16)
    return bits.reshape(m, -1)[:, :n] >= threshold(drop)
