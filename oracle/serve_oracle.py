"""fp64 oracle of running a quantized layer (include/pwq_serve.h): the
root-mean-square norm with residual and 8-bit output, the product with the
layer's codes, and the packed form's own definition.  numpy, shares no code
with the HIP path; test infrastructure only."""
import numpy as np


def rms_norm(x, weight, residual=None, eps=1e-6, eight_bit=False):
    """(y, step or None, codes or None, h): float64 [tokens, n]; with
    ``eight_bit`` the step max|y| / 127 (1 for a zero row) and rint(y / step)."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    if not eight_bit:
        return y, None, None, h
    step = np.max(np.abs(y), axis=1) / 127.0
    step = np.where(step == 0, 1.0, step)
    return y, step, np.rint(y / step[:, None]), h


def lattice_steps(codes, zeros, n):
    """c - z of every code, int64 [m, n]."""
    codes = np.asarray(codes, np.int64)
    if zeros is None:
        return codes
    z = np.asarray(zeros, np.int64)
    return codes - np.repeat(z, n // z.shape[1], axis=1)


def quantized_linear(x, codes, scales, zeros=None, x_scales=None):
    """(y, size): y = x W^^T in float64, and the sum of the terms' absolute
    values with |c - z| + 32 in place of c - z (what rounding errors scale
    with)."""
    x = np.asarray(x, np.float64)
    n = codes.shape[1]
    s = np.repeat(np.asarray(scales, np.float64), n // scales.shape[1], axis=1)
    step = lattice_steps(codes, zeros, n)
    y = x @ (s * step).T
    size = np.abs(x) @ (np.abs(s) * (np.abs(step) + 32)).T
    if x_scales is not None:
        xs = np.asarray(x_scales, np.float64)[:, None]
        y, size = y * xs, size * np.abs(xs)
    return y, size


def unpack(qweight, n, asym, outlier_off=None, outliers=None):
    """Codes int64 [m, n] of a packed layer, by the definition of its format."""
    q = np.asarray(qweight).astype(np.int64)
    m = q.shape[0]
    k = np.arange(n)
    half = (q[:, k // 2] >> (4 * (k % 2))) % 16
    codes = half if asym else np.where(half >= 8, half - 16, half)
    if outliers is not None:
        across = -(-n // 128)
        for tile in range(-(-m // 16) * across):
            for e in np.asarray(outliers)[outlier_off[tile]:outlier_off[tile + 1]].tolist():
                at = e & 0xffff
                codes[tile // across * 16 + at // 128, tile % across * 128 + at % 128] += e >> 16
    return codes
