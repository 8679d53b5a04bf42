"""MXFP4 / MXFP8 block quantization and the operators on it, in float64, from the
formats' definitions (tables of code values, ties to the even code); shares no
code with the library."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])  # code 127 is NaN


def _nearest(a, table):
    """Index of the table value nearest to a >= 0; ties to the even index; the
    largest value from above."""
    mid = (table[1:] + table[:-1]) / 2
    lo, hi = np.searchsorted(mid, a, "left"), np.searchsorted(mid, a, "right")
    return np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))


def quantize(v, table, top):
    """(codes [rows, cols] with the sign at bit log2(len(table) rounded up), scale
    bytes [rows, ceil(cols / 32)]) of the rows of v."""
    v = np.asarray(v, np.float64)
    rows, cols = v.shape
    nb = -(-cols // 32)
    b = np.zeros((rows, nb * 32))
    b[:, :cols] = v
    b = b.reshape(rows, nb, 32)
    amax = np.abs(b).max(-1)
    bad = ~np.isfinite(b).all(-1)
    safe = np.where(bad | (amax == 0), 1.0, amax)
    e = np.maximum(np.frexp(safe)[1] - 1 - top, -127)
    e = np.where(amax == 0, -127, e)
    scaled = np.where(bad[..., None], 0.0, np.ldexp(np.where(np.isfinite(b), b, 0.0), -e[..., None]))
    idx = _nearest(np.abs(scaled), table)
    sign = np.signbit(scaled).astype(np.int64) * (8 if len(table) == 8 else 128)
    codes = (idx + sign).reshape(rows, nb * 32)[:, :cols]
    return codes.astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def values(codes, scales, table):
    """The float64 values of codes and row-major scale bytes."""
    sbit = 8 if len(table) == 8 else 128
    mag = table[codes & (sbit - 1)]
    v = np.where(codes & sbit, -mag, mag)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=1)[:, :codes.shape[1]]


def qdq4(v):
    return values(*quantize(v, E2M1, 2), E2M1)


def qdq8(v):
    return values(*quantize(v, E4M3, 8), E4M3)


def pack(codes):
    """Codes as stored: two to a byte, rows of 64 * ceil(cols / 128) bytes."""
    rows, cols = codes.shape
    full = np.zeros((rows, -(-cols // 128) * 128), np.uint8)
    full[:, :cols] = codes
    return full[:, ::2] | (full[:, 1::2] << 4)


def tile(scales, cols):
    """Scale bytes as stored: tiles of 128 rows x 4 blocks."""
    rows = scales.shape[0]
    rt, kt = -(-rows // 128), -(-cols // 128)
    out = np.zeros(rt * kt * 512, np.uint8)
    for r in range(rows):
        for b in range(scales.shape[1]):
            out[((r // 128) * kt + b // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4] = \
                scales[r, b]
    return out


def silu_mul(g, u):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u


def ffn(x8, Wg, Wu, Wd):
    """One expert on rows that are quantized already; weights are float64 values."""
    return qdq8(silu_mul(x8 @ Wg.T, x8 @ Wu.T)) @ Wd.T


def layer(x, Wr, Wg, Wu, Wd, k, bias=None, shared=None, renorm=1):
    """y of the MXFP4 layer (unquantized weights given), and the chosen experts."""
    x = np.asarray(x, np.float64)
    lg = x @ Wr.T + (0 if bias is None else bias)
    ids = np.argsort(-lg, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(lg, ids, 1)
    w = np.exp(top - top[:, :1])
    w /= w.sum(1, keepdims=True) if renorm else np.exp(lg - top[:, :1]).sum(1, keepdims=True)
    x8 = qdq8(x)
    y = np.zeros_like(x)
    for e in range(Wr.shape[0]):
        t, r = np.nonzero(ids == e)
        if len(t):
            y[t] += w[t, r][:, None] * ffn(x8[t], qdq4(Wg[e]), qdq4(Wu[e]), qdq4(Wd[e]))
    if shared is not None:
        y += ffn(x8, *(qdq4(m) for m in shared))
    return y, ids
