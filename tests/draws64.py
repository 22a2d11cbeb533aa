"""The draws of dropout in plain integers, for the tests: Philox4x32-10 from its published definition."""
import numpy as np
import torch

M0, M1, W0, W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85


def philox(counter, key):
    """Ten rounds on four words (integers or uint64 arrays of 32-bit values) under two."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(v) for v in key]
    low, thirty_two = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        a, b = np.uint64(M0) * c[0], np.uint64(M1) * c[2]
        c = [(b >> thirty_two) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> thirty_two) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + W0) % 2 ** 32, (k[1] + W1) % 2 ** 32]
    return c


def cut_of(p):
    return int(np.floor(p * 65536 + 0.5))


def keep(rows, cols, p, seed, step, site, row0=0):
    """Which elements are kept, bool [rows, cols] on the CPU; row0: the first row's number."""
    groups = (cols + 7) // 8
    c0 = np.broadcast_to(np.arange(groups, dtype=np.uint64), (rows, groups))
    c1 = np.broadcast_to(np.arange(row0, row0 + rows, dtype=np.uint64)[:, None], (rows, groups))
    seed %= 2 ** 64
    w = philox((c0, c1, np.full((rows, groups), step % 2 ** 32), np.full((rows, groups), site)), (seed % 2 ** 32, seed >> 32))
    u = np.empty((rows, groups, 8), dtype=np.int64)
    for j in range(4):
        u[:, :, 2 * j] = w[j] & np.uint64(0xFFFF)
        u[:, :, 2 * j + 1] = w[j] >> np.uint64(16)
    return torch.from_numpy(u.reshape(rows, groups * 8)[:, :cols] >= cut_of(p))


def factor(p):
    """What a kept element is multiplied by."""
    return 65536.0 / (65536 - cut_of(p)) if cut_of(p) < 65536 else 0.0
