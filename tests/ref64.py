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


def round_bf16(v):
    """float64 -> nearest bf16 (ties to even), as float64.  The values met here are far inside bf16's range."""
    m, e = np.frexp(v)
    return np.ldexp(np.round(np.ldexp(m, 8)), e - 8)


def entering(v, wtype):
    """Activations v [rows, n] as a linear with weights of this type ("f32", "bf16", "fp8", "mxfp4") takes them."""
    if wtype == "mxfp4":
        return dequantize_mx(*quantize_mx(v, False), False)
    if wtype == "fp8":
        g = v.reshape(v.shape[0], -1, 128)
        s = np.abs(g).max(axis=-1, keepdims=True).astype(np.float32) * (np.float32(1) / np.float32(448))
        s = np.where(s == 0, np.float32(1), s)
        t = g.astype(np.float32) / s                      # the rule's fp32 quotient
        q = E4M3[nearest_code(np.minimum(np.abs(t), 448).astype(np.float64), E4M3)] * np.sign(t)
        return (q * s.astype(np.float64)).reshape(v.shape)
    return v


def weight(m, s, wtype):
    """float64 values of one stored matrix (numpy: fp32, bf16 bits, or bytes) and its scales."""
    if wtype == "mxfp4":
        return dequantize_mx(unpack(m), s, True)
    if wtype == "fp8":
        v = np.where(m & 128, -np.append(E4M3, np.nan)[m & 127], np.append(E4M3, np.nan)[m & 127])
        return v * np.repeat(np.repeat(s.astype(np.float64), 128, 0), 128, 1)
    if wtype == "bf16":
        return (m.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return m.astype(np.float64)


def expert(xq, m1, m3, m2, wtype):
    """A SwiGLU expert on rows xq (already as the first linears take them)."""
    act = (lambda v: v) if wtype == "f32" else round_bf16
    g, u = act(xq @ m1.T), act(xq @ m3.T)
    h = act(g / (1 + np.exp(-g)) * u)
    return act(entering(h, wtype) @ m2.T)


def layer(h, x, idx, w, wtype):
    """The layer for a given routing: h holds the stored weights by name (numpy), x [T, d] float64; y float64,
    not rounded at the end.  Slots outside [0, E) add nothing."""
    E = h["W1"].shape[0]
    one = lambda n, e: weight(h[n][e], None if h.get(n + "s") is None else h[n + "s"][e], wtype)   # noqa: E731
    xq = entering(x, wtype)
    y = expert(xq, *(weight(h[n], h.get(n + "s"), wtype) for n in ("S1", "S3", "S2")), wtype)
    for e in range(E):
        t, j = np.nonzero(idx == e)
        if len(t):
            np.add.at(y, t, expert(xq[t], one("W1", e), one("W3", e), one("W2", e), wtype) * w[t, j][:, None].astype(np.float64))
    return y
