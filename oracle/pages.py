"""Plain 64-bit forms of the calls that read less of a long cache: page bounds,
page scores, page selection and attention over given keys.  numpy only, one
row and head at a time, none of the library's code."""

import numpy as np

PAGE = 16


def bounds(k_cache, tables, lens, from_len=None, into=None):
    """[blocks][heads][2][dim] float64: least and greatest key of complete pages."""
    nb, hkv, _, d = k_cache.shape
    out = np.full((nb, hkv, 2, d), np.nan) if into is None else into.astype(np.float64).copy()
    for i, n in enumerate(lens):
        for t in range((0 if from_len is None else int(from_len[i])) // PAGE, int(n) // PAGE):
            b = tables[i, t]
            if 0 <= b < nb:
                out[b, :, 0], out[b, :, 1] = k_cache[b].min(axis=1), k_cache[b].max(axis=1)
    return out


def scores(q, bnd, table, n):
    """Of one row [heads][dim]: [kv heads][n] upper bounds, and the sums of the
    products' magnitudes (for an error bound)."""
    hkv = bnd.shape[1]
    group = q.shape[0] // hkv
    s, mag = np.zeros((hkv, n)), np.zeros((hkv, n))
    for g in range(hkv):
        for t in range(n):
            lo, hi = bnd[table[t], g]
            x = q[g * group:(g + 1) * group]
            best = np.maximum(x * lo, x * hi)
            s[g, t] = best.sum(1).max()
            mag[g, t] = np.abs(best).sum(1).max()
    return s, mag


def select(x, n, n_keep, n_first, n_last):
    """The pages of one row and head, ascending, then -1."""
    out = np.full(n_keep, -1, dtype=np.int32)
    if n <= n_keep:
        out[:n] = np.arange(n)
        return out
    keep = [t for t in range(n) if t < n_first or t >= n - n_last]
    value = [-np.inf if np.isnan(v) else float(v) for v in x[:n]]
    nan = [np.isnan(v) for v in x[:n]]
    rest = sorted((t for t in range(n) if n_first <= t < n - n_last), key=lambda t: (-value[t], nan[t], t))
    keep = sorted(keep + rest[:n_keep - len(keep)])
    out[:] = keep
    return out


def path(parent, j):
    """Local rows from j up to the root."""
    out = []
    while j >= 0:
        out.append(j)
        j = int(parent[j])
    return out


def attend_row(q, k_cache, v_cache, table, g, slots, scale):
    """Queries [heads of g][dim] over the cache slots: the output and the sums of
    the weighted magnitudes."""
    block, off = np.asarray([table[s // PAGE] for s in slots]), np.asarray(slots) % PAGE
    k, v = k_cache[block, g, off], v_cache[block, g, off]
    x = q @ k.T * scale
    w = np.exp(x - x.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    return w @ v, w @ np.abs(v)


def attend(q, k_cache, v_cache, tables, lens, cu, parent, windows, scale, cached):
    """All rows inside the windows: cached(i, r, g) are the context slots that row
    r (packed) sees by KV head g.  NaN where nothing is written."""
    out, mag = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    hkv = k_cache.shape[1]
    group = q.shape[1] // hkv
    for i, (b, e) in enumerate(windows):
        for j in range(b, e):
            r = cu[i] + j
            mine = [int(lens[i]) + m for m in path(parent[cu[i]:cu[i + 1]], j)]
            for g in range(hkv):
                h = slice(g * group, (g + 1) * group)
                out[r, h], mag[r, h] = attend_row(q[r, h], k_cache, v_cache, tables[i], g,
                                                  list(cached(i, r, g)) + mine, scale)
    return out, mag
