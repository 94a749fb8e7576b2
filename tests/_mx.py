"""The microscaled 4-bit format in plain numpy, in 64 bits: what the library's
zero_mx_* calls are tested against (host code only).

Quantising divides by a power of two and compares with the midpoints between
the format's magnitudes, both exact in float64, so codes and scales are
compared for equality; a midpoint goes to the even code."""
import numpy as np

BLOCK = 32
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
MID = (GRID[1:] + GRID[:-1]) / 2


def blocks(cols):
    return -(-cols // BLOCK)


def quantize(x):
    """[rows, cols] -> codes [rows, 16 * kb], scales [rows, kb], blocks along the rows."""
    x = np.asarray(x)
    rows, cols = x.shape
    kb = blocks(cols)
    v = np.zeros((rows, kb * BLOCK), dtype=np.float64)
    v[:, :cols] = x
    v = v.reshape(rows, kb, BLOCK)
    bad = ~np.isfinite(v).all(-1)
    v = np.where(bad[..., None], 0.0, v)
    amax = np.abs(v).max(-1, initial=0.0)
    e = np.frexp(amax)[1] - 1  # floor(log2)
    byte = np.where(amax > 0, np.maximum(e - 2, -127) + 127, 0)
    y = np.abs(v) / np.ldexp(1.0, byte - 127)[..., None]
    low, high = np.searchsorted(MID, y, side="left"), np.searchsorted(MID, y, side="right")
    mag = np.where(low % 2 == 0, low, high)  # they differ at a midpoint only
    code = (mag + 8 * np.signbit(v)).astype(np.uint8)
    code[bad] = 0
    code = code.reshape(rows, -1, 2)
    return code[..., 0] | (code[..., 1] << 4), np.where(bad, 255, byte).astype(np.uint8)


def decode(codes, scales):
    """codes [..., 16 * kb], scales [..., kb] -> float64 [..., 32 * kb] (NaN for NaN blocks)."""
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(*scales.shape, BLOCK)
    v = np.where(nib & 8, -1.0, 1.0) * GRID[nib & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (v * s[..., None]).reshape(*scales.shape[:-1], -1)


def product(a_codes, a_scales, b_codes, b_scales):
    """(sum_k a b, sum_k |a b|) in float64."""
    a, b = decode(a_codes, a_scales), decode(b_codes, b_scales)
    with np.errstate(invalid="ignore"):
        return a @ b.T, np.abs(a) @ np.abs(b).T


def random_mx(rng, rows, kb, lo=110, hi=140):
    """Random codes and scale bytes in [lo, hi)."""
    return (rng.integers(0, 256, (rows, 16 * kb), dtype=np.uint8),
            rng.integers(lo, hi, (rows, kb), dtype=np.int64).astype(np.uint8))
