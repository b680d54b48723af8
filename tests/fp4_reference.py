"""The 4-bit formats and operators in numpy, in 64 bits, from their definition
(include/qlinear.h): the reference of the 4-bit tests. Shares nothing with the
package; `unpack` reads codes and scale blocks byte by byte."""
import numpy as np

NV, MX = 0, 1
GROUP = {NV: 16, MX: 32}
_E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def _round_grid(y, man_bits, least_exp):
    """y >= 0 on a binary grid of man_bits fraction bits, ties to even."""
    _, e = np.frexp(y)
    step = np.exp2(np.maximum(e - 1, least_exp) - man_bits)
    return np.rint(y / step) * step


def e4m3_decode(b):
    b = b.astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * np.exp2(e - 7.0))
    return np.where((b & 127) == 127, np.nan, v)


def tensor_scale(x):
    a = np.abs(x.astype(np.float64)).max() if x.size else 0.0
    p = -80
    while 2688.0 * 2.0 ** p < a:
        p += 1
    return np.float32(2.0 ** p)


def scales(x, fmt, t=1.0):
    """Scale s of every group of the rows of x (float64), without t; NaN for a group with a non-finite element."""
    g = GROUP[fmt]
    m, k = x.shape
    n = -(-k // g)
    p = np.zeros((m, n * g))
    p[:, :k] = x
    with np.errstate(invalid="ignore"):
        amax = np.abs(p).reshape(m, n, g).max(-1)
    bad = ~np.isfinite(amax)
    amax = np.where(bad, 0.0, amax)
    if fmt == NV:
        # amax / (6 t) as fp32 computes it (6 t and the quotient rounded)
        d = (amax.astype(np.float32) / (np.float32(6) * np.float32(t))).astype(np.float64)
        s = _round_grid(np.clip(d, 2.0 ** -9, 448.0), 3, -6)
    else:
        f, e = np.frexp(amax / 6)
        s = np.exp2(np.clip(e - (f == 0.5), -127, 127).astype(np.float64))
        s[amax == 0] = 2.0 ** -127
    return np.where(bad, np.nan, s)


def quantise(x, fmt, t=1.0):
    """(E2M1 values, scales per element) of the rows of x [m, k]: value * scale is what x becomes."""
    x = x.astype(np.float64)
    m, k = x.shape
    s = np.repeat(scales(x, fmt, t), GROUP[fmt], axis=1)[:, :k]
    big = (s.astype(np.float32) * np.float32(t)).astype(np.float64) if fmt == NV else s
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        y = (x / big).astype(np.float32).astype(np.float64) if fmt == NV else x / big
        q = np.copysign(np.minimum(_round_grid(np.abs(y), 1, 0), 6.0), y)
    return np.where(np.isnan(s), 0.0, q), big


def values(x, fmt, t=1.0):
    q, s = quantise(x, fmt, t)
    return q * s


def unpack(q, sf, fmt, rows, cols, t=1.0, sf_rows=None, kcols=None):
    """Values [rows, cols] from codes [rows, bytes] and scale blocks, read by the layout alone. sf_rows: the
    row of the scale blocks of each row; kcols: columns that the scale blocks cover."""
    g = GROUP[fmt]
    kcols = cols if kcols is None else kcols
    words = -(-kcols // (4 * g))
    codes = np.zeros((rows, 2 * q.shape[1]), np.uint8)
    codes[:, 0::2], codes[:, 1::2] = q[:rows] & 15, q[:rows] >> 4
    codes = codes[:, :cols]
    mag = _E2M1[codes & 7]
    val = np.where(codes & 8, -mag, mag)
    r = (np.arange(rows) if sf_rows is None else np.asarray(sf_rows))[:, None]
    grp = (np.arange(cols) // g)[None, :]
    at = ((r // 128) * words + grp // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + grp % 4
    b = sf[at]
    if fmt == NV:
        s = (e4m3_decode(b).astype(np.float32) * np.float32(t)).astype(np.float64)
    else:
        s = np.where(b == 255, np.nan, np.exp2(b.astype(np.float64) - 127))
    return val * s


def expert_sf_rows(offsets):
    """Scale-block row of every row that an expert has (experts start on new 128-row blocks)."""
    out, base = {}, 0
    for a, b in zip(offsets[:-1], offsets[1:]):
        for r in range(a, b):
            out[r] = base + r - a
        base += -(-(b - a) // 128) * 128
    return out


def product(xv, wv):
    """X W^T and sum |x| |w| (for error bounds)."""
    return xv @ wv.T, np.abs(xv) @ np.abs(wv).T


def bound(absum, k):
    """Largest error of an fp32 product over k columns. Products of 4-bit values under 8-bit scales are exact in fp32;
    the sum is made in steps of 64 columns, each adding to an fp32 accumulator, and the last factors (two tensor scales,
    an accumulation into D) round once each: (k / 64 + 8) units of 2^-23 of sum |x| |w| allow a truncation at every step
    and eight more."""
    return (-(-k // 64) + 8) * 2.0 ** -23 * absum + 2.0 ** -148


def bf16(v):
    """float64 to the nearest bf16, ties to even (normal values)."""
    m, e = np.frexp(v)
    return np.ldexp(np.rint(m * 256), e - 8)
