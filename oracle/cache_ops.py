"""Oracle (test infrastructure only): what goes on around the attention over a
paged K/V cache, in float64 NumPy -- rotary positions with several axes, trees
of drafted tokens, the weight that attention gave to every cached row, and
which rows stay when a cache is cut down."""

import numpy as np


def rotate(x, pos, axis, freq):
    """Rows x [n][heads][dh] turned by their positions pos [axes][n]: pair j
    (elements j and j + len(freq)) by pos[axis[j]] * freq[j] radians."""
    x = np.asarray(x, np.float64)
    half = len(freq)
    y = x.copy()
    for j in range(half):
        a = np.asarray(pos[axis[j]], np.float64)[:, None] * freq[j]
        c, s = np.cos(a), np.sin(a)
        y[..., j] = x[..., j] * c - x[..., j + half] * s
        y[..., j + half] = x[..., j + half] * c + x[..., j] * s
    return y


def ancestors(parent):
    """[n][n] truth values: token t descends from token c, or is it."""
    n = len(parent)
    see = np.zeros((n, n), bool)
    for t, p in enumerate(parent):
        if 0 <= p < t:
            see[t] = see[p]
        see[t, t] = True
    return see


def tree_visible(see, kv_len):
    """[n][kv_len]: the keys that the drafted tokens see, the last n of the
    cache being their own."""
    n = len(see)
    out = np.ones((n, kv_len), bool)
    first = kv_len - n
    for t in range(n):
        for u in range(max(first, 0), kv_len):
            out[t, u] = see[t, u - first]
    return out


def mass(q, lse, k, pos, scale, right=-1):
    """One request: q [W][Hq][dh], lse [W][Hq], its cached rows k [L][H][dh], the
    rows' positions. Returns (weights summed per key and cached head [L][H], the
    same sums with every weight times what rounding can put it off by: the sum
    of |q||k| products in units of the last bit, and the exponent's size)."""
    W, Hq, dh = q.shape
    L, H, _ = k.shape
    g = Hq // H
    total, off = np.zeros((L, H)), np.zeros((L, H))
    see = np.ones((W, L), bool)
    if right >= 0:
        see = np.arange(L)[None] <= np.asarray(pos)[:, None] + right
    for h in range(Hq):
        s = scale * (q[:, h] @ k[:, h // g].T)
        mag = abs(scale) * (np.abs(q[:, h]) @ np.abs(k[:, h // g]).T)
        z = lse[:, h][:, None]
        some = see & np.isfinite(z)
        zz = np.where(np.isfinite(z), z, 0.0)
        w = np.where(some, np.exp(np.where(some, s - zz, 0.0)), 0.0)
        total[:, h // g] += w.sum(axis=0)
        off[:, h // g] += (w * ((dh + 8) * 2.0 ** -23 * mag + 2.0 ** -21 * (1 + np.abs(s) + np.abs(zz)))).sum(axis=0)
    return total, off


def keep(weights, budget, sinks, recent):
    """The positions that stay of weights [n], ascending."""
    n = len(weights)
    if n <= budget:
        return list(range(n))
    fixed = [u for u in range(n) if u < sinks or u >= n - recent]
    others = [u for u in range(n) if not (u < sinks or u >= n - recent)]
    rank = {u: (0 if np.isnan(weights[u]) else 1, 0.0 if np.isnan(weights[u]) else -weights[u], u) for u in others}
    return sorted(fixed + sorted(others, key=rank.get)[:budget - len(fixed)])
