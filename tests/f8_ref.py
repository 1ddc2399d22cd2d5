"""Plain 64-bit forms of the 8-bit base's operators (numpy), for the tests: quantising with a scale for
each block of 128, and products of 8-bit matrices.  No code of the library."""

import numpy as np

LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
FORMAT = {"e4m3": (3, -6), "e5m2": (2, -14)}  # bits of a significand, least exponent
TINY = 2.0 ** -64


def table(type):
    """The value of each of the 256 codes."""
    bits, low = FORMAT[type]
    code = np.arange(256)
    e, m = (code & 127) >> bits, code & ((1 << bits) - 1)
    v = np.where(e == 0, m * 2.0 ** (low - bits), (1 + m * 2.0 ** -bits) * 2.0 ** (np.maximum(e, 1) - 1.0 + low))
    if type == "e4m3":
        v[(code & 127) == 127] = np.nan
    else:
        v[(e == 31) & (m == 0)] = np.inf
        v[(e == 31) & (m > 0)] = np.nan
    return np.where(code > 127, -v, v)


def nearest(y, type):
    """The values nearest to y among a type's, ties to the even code, at most the largest."""
    bits, low = FORMAT[type]
    _, e = np.frexp(y)
    unit = np.ldexp(1.0, np.maximum(e - 1, low) - bits)
    with np.errstate(invalid="ignore"):
        return np.clip(np.round(y / unit) * unit, -LARGEST[type], LARGEST[type])


def quantize(x, block, type, pow2):
    """(values of the codes, scales) of fp32 values x."""
    rows, cols = x.shape
    rb, g = -(-rows // block), -(-cols // 128)
    codes, scales = np.zeros(x.shape), np.zeros((rb, g), dtype=np.float32)
    for i in range(rb):
        for j in range(g):
            at = (slice(i * block, (i + 1) * block), slice(j * 128, (j + 1) * 128))
            part = x[at].astype(np.float32)
            a = float(np.max(np.abs(part)))
            if a < TINY:
                continue
            if pow2 and np.isfinite(a):
                e = -140
                while LARGEST[type] * 2.0 ** e < a:
                    e += 1
                s = np.float32(2.0 ** e)
            else:
                s = np.float32(a) / np.float32(LARGEST[type])
            with np.errstate(invalid="ignore"):
                codes[at] = nearest((part / s).astype(np.float64), type)
            scales[i, j] = s
    return codes, scales


def widen(codes, scales, block):
    """Values of a matrix from its codes' and its scales, in doubles."""
    rows, cols = codes.shape
    return codes * scales.astype(np.float64)[np.arange(rows) // block][:, np.arange(cols) // 128]
