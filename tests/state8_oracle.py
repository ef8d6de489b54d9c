"""The block-scaled 8-bit states and the steps over lists of tensors, in numpy, from the
definitions in include/zero.h: fp32 where the definition says fp32, so codes can be
compared bit for bit, and 64-bit twins of the formulas for the tolerances."""
import numpy as np

BLOCK = 256
NEAREST = np.uint32(1 << 19)
M32 = np.uint64(0xFFFFFFFF)


def _mix(x):
    x = np.asarray(x, np.uint64) & M32
    x = x ^ (x >> np.uint64(16))
    x = x * np.uint64(0x6A09E667) & M32
    x = x ^ (x >> np.uint64(15))
    x = x * np.uint64(0xBB67AE85) & M32
    return x ^ (x >> np.uint64(16))


def random20(n_blocks, seed, t, block0, name):
    """The 20 random bits of every element of n_blocks blocks, the first being block0."""
    lo, hi = np.uint64(seed & 0xFFFFFFFF), np.uint64(seed >> 32)
    key = _mix(_mix((lo + np.uint64(t * 0x9E3779B9 & 0xFFFFFFFF)) & M32) ^ hi)
    g = np.arange(block0 * 32, (block0 + n_blocks) * 32, dtype=np.uint64)
    s = _mix(key + (g * np.uint64(0x9E3779B9) & M32))
    out = np.empty((g.size, 8), np.uint32)
    for j in range(1, 17):
        s = (s * np.uint64(1664525) + np.uint64(1013904223)) & M32
        k = j - (1 if name == "m" else 9)
        if 0 <= k < 8:
            out[:, k] = s >> np.uint64(12)
    return out.reshape(-1)


def _blocks(x, fill=0):
    n = -(-x.size // BLOCK) * BLOCK
    return np.concatenate([x, np.full(n - x.size, fill, x.dtype)]).reshape(-1, BLOCK)


def exponents(x):
    top = np.abs(_blocks(x)).max(1) if x.size else np.zeros(0, np.float32)
    bits = np.minimum(top.view(np.uint32), np.uint32(0x7F800000)).astype(np.int64)
    b = np.clip((bits + 0xFFFFF) >> 23, 27, 253)
    return np.where(top == 0, 0, b).astype(np.int64)


def encode(x, name, r):
    """(codes, exponents) of fp32 x; r: a 20-bit addend, or one per element of the blocks."""
    b = exponents(x)
    e = np.repeat(b, BLOCK)[:x.size]
    up = ((254 - e) << 23).astype(np.uint32).view(np.float32)
    y = (np.abs(x) * up) * np.float32(2.0 ** (-112 if name == "m" else -96))
    r = np.asarray(r, np.uint32)
    r = r[:x.size] if r.ndim else r
    c = (y.view(np.uint32).astype(np.int64) + r.astype(np.int64)) >> 20
    if name == "m":
        return (np.minimum(c, 127) | (x.view(np.uint32) >> 24 & 0x80)).astype(np.uint8), b
    return np.maximum(np.minimum(c, 255), x > 0).astype(np.uint8), b


def decode(c, b, name):
    e = np.repeat(np.asarray(b, np.int64), BLOCK)[:c.size]
    mag = (c.astype(np.uint32) & (0x7F if name == "m" else 0xFF)) << np.uint32(20)
    y = mag.view(np.float32) * np.float32(2.0 ** (112 if name == "m" else 96))
    y = y * (e.astype(np.uint32) << np.uint32(23)).view(np.float32)
    return np.where(c & 0x80, -y, y).astype(np.float32) if name == "m" else y


def moments(x, m, v, c, inv, b1, b2, dtype=np.float32):
    f = dtype
    b1, b2, one = np.float32(b1), np.float32(b2), np.float32(1)
    o1, o2 = f(one - b1), f(one - b2)
    gc = f(np.float32(c)) * (x.astype(f) * f(np.float32(inv)))
    return f(b1) * m.astype(f) + o1 * gc, f(b2) * v.astype(f) + o2 * (gc * gc)


def update(p, m, v, step, rbc2, decay, eps, dtype=np.float64):
    f = dtype
    denom = np.sqrt(v.astype(f)) / f(np.float32(rbc2)) + f(np.float32(eps))
    return p.astype(f) * f(np.float32(decay)) - f(np.float32(step)) * (m.astype(f) / denom)
