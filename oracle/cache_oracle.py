"""fp64 oracle of the key-value cache (include/pwq_cache.h): the quantization of
a head, the layout of a record, and attention.  numpy, shares no code with the
HIP path; test infrastructure only."""
import numpy as np


def quantize(x, bits):
    """(codes int64, steps float32, zero points int64) of x [..., D], float32 values."""
    x = np.asarray(x, np.float32).astype(np.float64)
    top = 2 ** bits - 1
    bad = ~np.isfinite(x).all(-1)
    safe = np.where(bad[..., None], 0.0, x)
    lo, hi = np.minimum(safe.min(-1), 0), np.maximum(safe.max(-1), 0)
    with np.errstate(over="ignore"):
        span = (hi - lo).astype(np.float32)                  # both fit 53 bits, or it is far off
    bad |= ~np.isfinite(span)
    span = np.where(bad, np.float32(0), span)
    step = (span.astype(np.float64) / top).astype(np.float32)
    step = ((step.view(np.uint32) + np.uint32(128)) & np.uint32(0xFFFFFF00)).view(np.float32)
    s = np.where(step == 0, 1.0, step.astype(np.float64))
    z = np.where(step == 0, 0, np.minimum(np.rint(-lo / s), top))
    c = np.clip(np.rint(safe / s[..., None]) + z[..., None], 0, top)
    c = np.where((step == 0)[..., None], 0, c)
    return (c.astype(np.int64), np.where(bad, np.float32(np.nan), step),
            np.where(bad, 0, z).astype(np.int64))


def values(codes, steps, zeros):
    return np.asarray(steps, np.float64)[..., None] * (codes - zeros[..., None])


def record_bytes(dim, bits):
    return 8 * dim * bits + 256


def key_bit(p, d, dim, bits):
    """Bit of a record where the code of token p's key channel d starts."""
    t, a = divmod(p, 16)
    j, rest = divmod(d, 32)
    g, e = divmod(rest, 8)
    n = (t * (dim // 32) + j) * bits                         # bytes of the lane before (t, j)
    bit = 8 * n + (8 * e if bits == 8 else 4 * (e // 2) + 16 * (e % 2))
    return _lane_bit(16 * g + a, bit)


def value_bit(p, d, dim, bits):
    t, rest = divmod(p, 16)
    g, i = divmod(rest, 4)
    n, a = divmod(d, 16)
    unit = n if bits == 8 else n // 2
    bit = 8 * (unit * 8 + 4 * t + i) + (4 * (n % 2) if bits == 4 else 0)
    return 8 * 4 * dim * bits + _lane_bit(16 * g + a, bit)


def _lane_bit(lane, bit):
    byte = bit // 8
    return 8 * (byte // 16 * 1024 + lane * 16 + byte % 16) + bit % 8


def bit_table(dim, bits):
    """int64 [2, 32, dim]: where every code of a record starts."""
    return np.array([[[f(p, d, dim, bits) for d in range(dim)] for p in range(32)]
                     for f in (key_bit, value_bit)])


def unpack(records, dim, bits):
    """(codes, steps, zeros) of records [..., bytes]: [..., 2, 32, dim], [..., 2, 32]."""
    r = np.asarray(records, np.uint8)
    at = bit_table(dim, bits)
    codes = (r[..., at // 8].astype(np.int64) >> (at % 8)) % 2 ** bits
    words = np.ascontiguousarray(r[..., 8 * dim * bits:]).view(np.uint32)
    words = words.reshape(*r.shape[:-1], 2, 32)
    return (codes, (words & np.uint32(0xFFFFFF00)).view(np.float32),
            (words & np.uint32(255)).astype(np.int64))


def pack(codes, steps, zeros, dim, bits):
    """Records [..., bytes] of codes [..., 2, 32, dim]."""
    lead = codes.shape[:-3]
    at = bit_table(dim, bits)
    r = np.zeros((*lead, record_bytes(dim, bits)), np.uint8)
    for of in range(2):
        for p in range(32):
            for d in range(dim):
                b = at[of, p, d]
                r[..., b // 8] |= (codes[..., of, p, d] << (b % 8)).astype(np.uint8)
    words = np.asarray(steps, np.float32).view(np.uint32) | zeros.astype(np.uint32)
    r[..., 8 * dim * bits:] = np.ascontiguousarray(words).view(np.uint8).reshape(*lead, 256)
    return r


def stored(records, table, length, dim, bits, page):
    """Keys and values float64 [heads, length, dim] of a sequence's tokens, and
    whether they are there (not holes): bool [length]."""
    pages, heads = records.shape[:2]
    out = np.zeros((2, heads, length, dim))
    there = np.zeros(length, bool)
    for first in range(0, length, 32):
        entry = first // page
        if entry >= len(table) or not 0 <= table[entry] < pages:
            continue
        vals = values(*unpack(records[table[entry], :, first % page // 32], dim, bits))
        n = min(32, length - first)
        out[:, :, first:first + n] = vals.transpose(1, 0, 2, 3)[:, :, :n]
        there[first:first + n] = True
    return out[0], out[1], there


def attention(q, k, v, scale, seen):
    """(out, size, score) for one head: q [rows, D], k, v [tokens, D], seen bool
    [rows, tokens]; size = sum w |v| (what rounding errors of weights scale with),
    score = the largest scale * sum |q| |k| of a row."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    s = np.where(seen, scale * (q @ k.T), -np.inf)
    top = np.where(seen.any(1), s.max(1, initial=-np.inf), 0.0)
    w = np.exp(s - top[:, None])
    total = w.sum(1, keepdims=True)
    w = w / np.where(total == 0, 1, total)
    size = w @ np.abs(v)
    score = np.where(seen, scale * (np.abs(q) @ np.abs(k).T), 0).max(1, initial=0)
    return w @ v, size, score
