"""AdamW in numpy, element by element from its definition: in 64 bits, and in 32 bits with every
product and sum rounded on its own, which is what decides the 8-bit codes."""
import numpy as np

BLOCK = 256
_MASK = (1 << 64) - 1


def _mix(z):
    z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
    z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
    return z ^ (z >> np.uint64(31))


def random_bits(seed, step, tensor, n):
    """The 16 bits that round m and the 16 that round v, for n elements."""
    key = _mix(np.array([(seed + step * 2654435769) & _MASK], np.uint64))
    key = _mix(key + np.uint64(tensor))
    z = _mix(key + np.uint64(0x9E3779B97F4A7C15) * (np.arange((n + 1) // 2, dtype=np.uint64) + np.uint64(1)))
    half = np.stack([z & np.uint64(0xFFFFFFFF), z >> np.uint64(32)], 1).reshape(-1)[:n].astype(np.int64)
    return half & 0xFFFF, half >> 16


def value_table(bias, n):
    """The value of each code: f 2^(-bias-2) below 8, else (1 + f/8) 2^(e-bias)."""
    return np.array([(1 + (c % 8) / 8) * 2.0 ** (c // 8 - bias) if c >= 8 else c * 2.0 ** (-2 - bias) for c in range(n)])


E4M3, U53 = value_table(7, 128), value_table(15, 256)


def decode(codes, scales, kind):
    c = codes.astype(np.int64)
    if kind == "m":
        v = np.where(c & 128, -1.0, 1.0) * E4M3[c & 127]
    else:
        v = U53[c]
    return v.astype(np.float32) * np.repeat(scales.astype(np.float32), BLOCK)[:c.size]


def encode(x, u, kind):
    """(codes, scales) of float32 values, by floor(distance / spacing + u / 2^16) in exact integers."""
    top, table, most = (448.0, E4M3, 0x7E) if kind == "m" else (61440.0, U53, 0xF7)
    n = x.size
    pad = np.zeros(-(-n // BLOCK) * BLOCK, np.float32)
    pad[:n] = np.abs(x)
    big = pad.reshape(-1, BLOCK).max(1)
    dead = big < np.float32(2.0 ** -100)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        inv = np.where(dead, np.float32(0), np.float32(top) / big).astype(np.float32)
        scales = np.where(dead, np.float32(0), big / np.float32(top)).astype(np.float32)
        y = np.abs(x) * np.repeat(inv, BLOCK)[:n]
    low = np.searchsorted(table[:most + 1], np.minimum(y, top), side="right") - 1
    spacing = np.where(low < 8, table[1], 2.0 ** (np.floor(np.log2(np.maximum(table[low], table[1]))) - 3))
    spacing = np.maximum(spacing, table[1])
    left = (y.astype(np.float64) - table[low]) / spacing  # exact: both are binary fractions of the spacing
    # below the normal range the kernel adds in 32 bits: y / spacing + u / 2^16, rounded, then floor
    small = y < 8 * table[1]
    s = ((y * np.float32(1 / table[1])) + (u.astype(np.float32) * np.float32(2.0 ** -16))).astype(np.float32)
    up = np.where(small, np.floor(s) > low, left * 65536 + u >= 65536)
    codes = np.minimum(low + up, most)
    if kind == "v":
        codes = np.where((x > 0) & (codes == 0) & ~np.repeat(dead, BLOCK)[:n], 1, codes)
    else:
        codes = codes | np.where(np.signbit(x), 128, 0)
    return codes.astype(np.uint8), scales


def step(p, g, m, v, t, lr, betas, eps, decay, clip, dtype):
    """One step in `dtype` (np.float64, or np.float32 with each operation rounded)."""
    f = dtype
    b1, b2 = betas
    p, g, m, v = (a.astype(f) for a in (p, g, m, v))
    g = g * f(clip)
    m = m * f(b1) + g * f(1 - b1)
    v = v * f(b2) + (g * f(1 - b2)) * g
    p64, m64, v64 = (a.astype(np.float64) for a in (p, m, v))
    with np.errstate(divide="ignore", invalid="ignore"):
        p = p64 * (1 - lr * decay) - lr * (m64 / (1 - b1 ** t)) / (np.sqrt(v64 / (1 - b2 ** t)) + eps)
    return p, m, v
