"""The decoder-layer operators in fp64 numpy: rotation and appending to a paged cache, attention over shared prefixes,
products with a 4-bit matrix.  Written from the formulas; used by tests only."""
import numpy as np


# ------------------------------------------------------------------- e4m3
def e4m3_value(code):
    """fp64 values of e4m3 codes (uint8): sign, 4 exponent bits (bias 7), 3 mantissa bits, no infinity, NaN at 0x7F."""
    c = np.asarray(code, np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


_POSITIVE = e4m3_value(np.arange(127))


def e4m3_code(x):
    """The nearest code of each value, ties to the even code, saturated at +-448; NaN stays NaN."""
    a = np.minimum(np.abs(np.asarray(x, np.float64)), 448.0)
    hi = np.clip(np.searchsorted(_POSITIVE, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _POSITIVE[lo], _POSITIVE[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(np.isnan(x), 127, c)
    return (c | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


# --------------------------------------------------------------- rotation
def rotate(x, pos, inv_freq, interleaved):
    """x [n][heads][dim] with the first 2 len(inv_freq) elements of each head rotated by pos * inv_freq."""
    y = np.array(x, np.float64)
    f = np.asarray(inv_freq, np.float64)
    i = np.arange(f.size)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + f.size)
    ang = np.asarray(pos, np.float64)[:, None, None] * f
    u, v = y[..., a].copy(), y[..., b].copy()
    y[..., a] = u * np.cos(ang) - v * np.sin(ang)
    y[..., b] = v * np.cos(ang) + u * np.sin(ang)
    return y


# -------------------------------------------------------------- attention
def gather(pool, table, n, page):
    """The first n rows of a sequence: pool [pages][heads][page][dim] -> [n][heads][dim]."""
    pool = np.asarray(pool, np.float64)
    i = np.arange(n)
    return pool[np.asarray(table)[i // page], :, i % page]


def attend(q, k, v, visible, scale):
    """One sequence: q [n][hq][d], k and v [m][hkv][d], visible [n][m].  Returns (y, spread, size) [n][hq][d] with
    y = sum w v, spread = sum w |v - y|, size = sum w |v| for the softmax weights w over the visible keys (all zero
    for a row that sees none), and reach [n][hq] = the largest sum_i |q_i k_i| of a visible key."""
    n, hq, d = q.shape
    r = hq // k.shape[1]
    y, spread, size = (np.zeros((n, hq, d)) for _ in range(3))
    reach = np.zeros((n, hq))
    for t in range(n):
        see = np.nonzero(visible[t])[0]
        if not see.size:
            continue
        for h in range(hq):
            kk, vv = k[see, h // r], v[see, h // r]
            s = (kk @ q[t, h]) * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            y[t, h] = w @ vv
            spread[t, h] = w @ np.abs(vv - y[t, h])
            size[t, h] = w @ np.abs(vv)
            reach[t, h] = (np.abs(kk) @ np.abs(q[t, h])).max()
    return y, spread, size, reach


# ------------------------------------------------------------------ 4-bit
def w4_pack(codes, scale, zero):
    """Bytes of the 4-bit format: codes [out][in] (0..15), scale and zero fp16 [in/128][out]."""
    out, inn = codes.shape
    words = np.zeros((out // 16, inn // 128, 4, 16, 4), np.uint32)
    for e in range(8):
        sub = codes.reshape(out // 16, 16, inn // 128, 4, 4, 8)[..., e].transpose(0, 2, 3, 1, 4)
        words |= sub.astype(np.uint32) << np.uint32(4 * (e // 2) + 16 * (e % 2))
    sz = np.asarray(scale, np.float16).view(np.uint16).astype(np.uint32) | \
        (np.asarray(zero, np.float16).view(np.uint16).astype(np.uint32) << np.uint32(16))
    return np.concatenate([words.reshape(-1), sz.reshape(-1)]).view(np.uint8)


def w4_matrix(codes, scale, zero):
    """The fp64 matrix that the format stands for."""
    rep = lambda a: np.repeat(np.asarray(a, np.float64).T, 128, axis=1)  # noqa: E731
    return rep(scale) * (codes.astype(np.float64) - rep(zero))
