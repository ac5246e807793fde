"""Plain 64-bit forms of the microscaled formats and of the layer for a given routing, on the CPU (numpy),
written from the definitions in include/moe.h for the tests of those operators."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
_c = np.arange(127)
E4M3 = np.where(_c >> 3 == 0, (_c & 7) / 8 * 2.0 ** -6, (1 + (_c & 7) / 8) * 2.0 ** ((_c >> 3) - 7.0))   # codes 0 .. 126


def nearest_code(a, grid):
    """Index of the value of `grid` (ascending from 0) nearest to a >= 0; a tie goes to the even index."""
    mid = (grid[1:] + grid[:-1]) / 2                     # exact: neighbours differ by a power of two
    lo = np.searchsorted(mid, a, side="left")            # at a midpoint: the lower neighbour
    tie = (lo < len(mid)) & (a == mid[np.minimum(lo, len(mid) - 1)]) & (lo % 2 == 1)
    return (lo + tie).astype(np.uint8)


def quantize_mx(x, fp4):
    """(codes one to a byte with the sign on top, scale codes) of x [rows, cols] float64; non-finite groups as
    the library defines them."""
    rows, cols = x.shape
    g = x.reshape(rows, cols // 32, 32)
    amax = np.abs(g).max(axis=-1)
    bad = ~np.isfinite(g).all(axis=-1)
    _, e = np.frexp(np.where(bad, 1.0, amax))            # amax = m 2^e, m in [1/2, 1): floor(log2) = e - 1
    se = np.clip(e - 1 - (2 if fp4 else 8), -127, 127)
    se = np.where(amax == 0, -127, se)
    t = np.ldexp(np.where(bad[..., None], 0.0, g), -se[..., None])
    q = nearest_code(np.abs(t), E2M1 if fp4 else E4M3)
    q = np.where(np.signbit(t), q | (8 if fp4 else 128), q)
    q = np.where(bad[..., None], 0, q).astype(np.uint8)
    return q.reshape(rows, cols), np.where(bad, 255, se + 127).astype(np.uint8)


def dequantize_mx(q, scales, fp4):
    """float64 values of codes [rows, cols] (one to a byte) with scale codes [rows, cols / 32]."""
    if fp4:
        v = np.where(q & 8, -E2M1[q & 7], E2M1[q & 7])
    else:
        grid = np.append(E4M3, np.nan)
        v = np.where(q & 128, -grid[q & 127], grid[q & 127])
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def pack(q):
    """E2M1 codes [..., cols] -> bytes [..., cols / 2], the lower column in the low half."""
    return (q[..., 0::2] | (q[..., 1::2] << 4)).astype(np.uint8)


def unpack(b):
    return np.stack([b & 15, b >> 4], axis=-1).reshape(*b.shape[:-1], -1)
