"""Reference of the counter-based dropout mask: Philox4x32-10 (Salmon et al.,
SC 2011) in numpy 64-bit integers, one counter (block of eight elements,
offset) per row."""
import numpy as np
import torch

M32 = (1 << 32) - 1


def philox(ctr, key):
    """ctr: uint64 array [n, 4] of 32-bit words; key: two 32-bit ints."""
    c = [np.asarray(ctr[:, i], np.uint64) for i in range(4)]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(10):
        p0 = c[0] * np.uint64(0xD2511F53)
        p1 = c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), p1 & np.uint64(M32),
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p0 & np.uint64(M32)]
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    return np.stack(c, 1).astype(np.uint32)


def halves(n, seed, offset, first=0):
    """The 16-bit halves of elements [first, first + n) (first % 8 == 0)."""
    assert first % 8 == 0
    blk = np.arange(first // 8, (first + n + 7) // 8, dtype=np.uint64)
    ctr = np.stack([blk & np.uint64(M32), blk >> np.uint64(32),
                    np.full_like(blk, offset & M32), np.full_like(blk, (offset >> 32) & M32)], 1)
    w = philox(ctr, (seed & M32, seed >> 32))
    return np.stack([w & 0xFFFF, w >> 16], 2).reshape(-1)[:n]


def threshold(p):
    return int(np.floor(float(np.float32(p)) * 65536 + 0.5))


def scale(p):
    return np.float32(65536) / np.float32(65536 - threshold(p))


def keep(shape, p, seed, offset, first=0):
    """bool tensor (CPU): True where the element is kept."""
    n = int(np.prod(shape))
    return torch.from_numpy(halves(n, seed, offset, first) >= threshold(p)).view(*shape)


def drop_f32(x, p, seed, offset, first=0):
    """Dropout of a CPU tensor in float32, as the kernels form it before
    rounding: one float32 product per kept element, +0 elsewhere."""
    k = keep(x.shape, p, seed, offset, first)
    return torch.where(k, x.float() * float(scale(p)), torch.zeros(()))
