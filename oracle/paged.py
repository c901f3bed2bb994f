"""Oracle (test infrastructure only): the paged K/V cache in float64 NumPy.

A cached row of one head holds its elements as bf16 or, in 8 bits, as e4m3
codes with one power-of-two scale: the row stands for code * 2^e with the
least e >= -117 for which max|x| <= 448 * 2^e; a row with an infinity or NaN
stands for NaN. Attention over the cache: a
query row at position p sees the cached positions u < kv_len with
u <= p + right, and with u >= p - left or u < sinks.
"""

import numpy as np

E_MIN = -117


def _code_values():
    """The value of every e4m3 code (sign, 4 exponent bits with bias 7, 3
    mantissa bits; no infinities, S.1111.111 is NaN)."""
    c = np.arange(256)
    s, e, m = np.where(c & 0x80, -1.0, 1.0), (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e.astype(np.float64) - 7))
    v = s * v
    v[(c & 0x7F) == 0x7F] = np.nan
    return v


E4M3 = _code_values()


def nearest_code(x):
    """The e4m3 code nearest to each x, |x| <= 448 (ties to the even mantissa)."""
    pos = E4M3[:0x7F]                                    # increasing, codes 0 .. 0x7E
    a = np.abs(x)
    hi = np.clip(np.searchsorted(pos, a), 1, 0x7E)
    lo = hi - 1
    d_lo, d_hi = a - pos[lo], pos[hi] - a
    code = np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi)
    return np.where(np.signbit(x), code | 0x80, code).astype(np.uint8)


def quantise(x):
    """(codes uint8, scale bytes uint8) of rows x [..., dh] of bf16 values. A
    row with an infinity or NaN has the byte 255 (its codes mean nothing: 0
    here)."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x).all(axis=-1)
    x = np.where(fine[..., None], x, 0.0)
    top = np.abs(x).max(axis=-1)
    e = np.full(top.shape, E_MIN)
    for k in range(E_MIN, 121):
        e = np.where(top > 448 * 2.0 ** e, k + 1, e)
    lim = np.where(e == 120, 240.0, 448.0)[..., None]     # a code may not stand for 2^128
    codes = nearest_code(np.clip(x / (2.0 ** e)[..., None], -lim, lim))
    return codes, np.where(fine, e + 127, 255).astype(np.uint8)


def restore(codes, scale):
    """The values that codes [..., dh] with scale bytes [...] stand for."""
    f = np.where(scale == 255, np.nan, 2.0 ** (np.minimum(scale, 254).astype(np.float64) - 127))
    return E4M3[codes] * f[..., None]


def visible(pos, kv_len, left, right, sinks):
    """[len(pos)][kv_len] truth values: which keys the rows at `pos` see."""
    u, p = np.arange(kv_len)[None], np.asarray(pos)[:, None]
    see = np.ones((len(pos), kv_len), bool)
    if right >= 0:
        see &= u <= p + right
    if left >= 0:
        see &= (u >= p - left) | (u < sinks)
    return see


def attention(q, k, v, pos, scale, left=-1, right=-1, sinks=0, see=None):
    """One request: q [W][Hq][dh], its cached rows k, v [L][H][dh], the rows'
    positions [W], or what they see as truth values `see` [W][L]. Returns (out, lse, weighted |v| sums, score magnitudes):
    the last two are what rounding of the weights and of the scores scales
    with. What no row sees is not read."""
    W, Hq, dh = q.shape
    L, H, _ = k.shape
    see = visible(pos, L, left, right, sinks) if see is None else see
    used = see.any(axis=0)
    out, lse = np.zeros((W, Hq, dh)), np.full((W, Hq), -np.inf)
    absv, mag = np.zeros((W, Hq, dh)), np.zeros((W, Hq))
    for h in range(Hq):
        kh = np.where(used[:, None], k[:, h * H // Hq], 0.0)
        vh = np.where(used[:, None], v[:, h * H // Hq], 0.0)
        s = np.where(see, scale * (q[:, h] @ kh.T), -np.inf)
        m = s.max(axis=1, initial=-np.inf)
        some = m > -np.inf
        p = np.exp(s - np.where(some, m, 0.0)[:, None])
        z = p.sum(axis=1)
        zz = np.where(some, z, 1.0)
        out[:, h] = (p @ vh) / zz[:, None]
        absv[:, h] = (p @ np.abs(vh)) / zz[:, None]
        lse[some, h] = m[some] + np.log(z[some])
        mag[:, h] = np.where(see, abs(scale) * (np.abs(q[:, h]) @ np.abs(kh).T), 0.0).max(axis=1, initial=0.0)
    return out, lse, absv, mag
