"""fp64 oracle of MXFP4 (E2M1 codes, one E8M0 scale per 32): quantiser, values, and the layer's products with such
weights.  Written from the format's definition; imports nothing from the package.

E2M1: sign, 2 exponent bits (bias 1), 1 mantissa bit, no infinities and no NaN: 0, 0.5, 1, 1.5, 2, 3, 4, 6.
    X = floor(log2 amax) - 2 (2 = exponent of the largest value), clamped to -127; all-zero block -> -127
    code = RNE_E2M1(clamp(v / 2^X, -6, 6)), ties to the even code;  scale byte = X + 127
A block that holds an infinity or a NaN has the scale byte 255 (NaN)."""
from __future__ import annotations

import numpy as np

VALUES = np.array([(m / 2.0 if e == 0 else (1 + m / 2.0) * 2.0 ** (e - 1)) for e in range(4) for m in range(2)])
TABLE = np.concatenate([VALUES, -VALUES])


def encode(v):
    """Codes 0..15 of already scaled values: a search of the nearest value, the sign kept also for zero."""
    a = np.minimum(np.abs(np.asarray(v, dtype=np.float64)), 6.0)
    d = np.abs(a[..., None] - VALUES)
    near = d == d.min(axis=-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(axis=-1), even.argmax(axis=-1), near.argmax(axis=-1))
    return (code + 8 * np.signbit(v)).astype(np.uint8)


def quantise(v):
    """(codes [N, K], scale bytes [N, K / 32]) of fp64 rows."""
    N, K = v.shape
    b = v.reshape(N, K // 32, 32)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[:, :, None], 0.0, b)
    amax = np.abs(b).max(axis=2)
    X = np.where(amax > 0, np.frexp(amax)[1] - 3, -127).clip(-127, 127)
    c = encode(np.ldexp(b, -X[:, :, None])).reshape(N, K)
    c[np.repeat(bad, 32, axis=1)] = 0
    return c, np.where(bad, 255, X + 127).astype(np.uint8)


def unpack(codes):
    """[N, K / 2] bytes -> codes [N, K]: the even column in the low half."""
    return np.stack([codes & 15, codes >> 4], axis=-1).reshape(codes.shape[0], -1)


def scale_rows(scales):
    """The layout [K / 128][N][4] as [N, K / 32]."""
    return np.ascontiguousarray(scales.transpose(1, 0, 2)).reshape(scales.shape[1], -1)


def values(codes, scales):
    """fp64 matrix of packed codes [N, K / 2] and scales [K / 128][N][4]."""
    s = scale_rows(scales).astype(np.int64)
    f = np.where(s == 255, np.nan, np.ldexp(1.0, np.minimum(s, 254) - 127))
    return TABLE[unpack(codes)] * np.repeat(f, 32, axis=1)


def swiglu(a, u):
    with np.errstate(over="ignore"):
        return a / (1.0 + np.exp(-a)) * u
