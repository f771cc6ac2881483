"""The paged key/value cache and the attention of drafted rows over it, in fp64 — test infrastructure only.

Every function takes NumPy arrays.  A cache is a dict: k, v [n_pages, heads, page, D] (the values codes stand for before
their scales), k_scale, v_scale [n_pages, heads, page] or None, table [n_req, max_pages].
"""
import numpy as np

from .vocab import AMAX_MIN, e4m3_round


def place(cache: dict, r: int, pos: int):
    """(page, slot) of a position, None where there is none."""
    n_pages, _, size, _ = cache["k"].shape
    table = cache["table"]
    if not (0 <= r < table.shape[0] and 0 <= pos < table.shape[1] * size):
        return None
    page = int(table[r, pos // size])
    return (page, pos % size) if 0 <= page < n_pages else None


def quant_row(x):
    """(quotients before rounding to e4m3, scale) of rows [..., D]; a non-finite element is NaN."""
    fin = np.isfinite(x)
    amax = np.maximum(np.abs(np.where(fin, x, 0.0)).max(-1), AMAX_MIN)
    return np.where(fin, x, np.nan) * (448.0 / amax)[..., None], amax / 448.0


def write(cache: dict, k, v, mark_req, mark_pos, base, n: int, to_bf16=None) -> tuple:
    """Writes in place; returns the rows that had no place.  to_bf16 rounds for a cache without scales."""
    bad = []
    for i in range(n):
        r = int(mark_req[i])
        if r == -1:
            continue
        at = place(cache, r, int(base[r]) + int(mark_pos[i])) if 0 <= r < len(base) else None
        if at is None:
            bad.append(i)
            continue
        for name, x in (("k", k[i]), ("v", v[i])):
            if cache[name + "_scale"] is None:
                cache[name][at[0], :, at[1]] = to_bf16(x)
            else:
                q, s = quant_row(x)
                cache[name][at[0], :, at[1]] = np.where(np.isnan(q), np.nan, e4m3_round(np.nan_to_num(q)))
                cache[name + "_scale"][at[0], :, at[1]] = s
    return bad


def rows(cache: dict, name: str, r: int, positions) -> np.ndarray:
    """[len(positions), heads, D] in fp64; NaN where a position has no place."""
    _, heads, _, D = cache[name].shape
    out = np.full((len(positions), heads, D), np.nan)
    for n, pos in enumerate(positions):
        at = place(cache, r, int(pos))
        if at is not None:
            out[n] = cache[name][at[0], :, at[1]]
            if cache[name + "_scale"] is not None:
                out[n] *= cache[name + "_scale"][at[0], :, at[1]][:, None]
    return out


def move(cache: dict, base, path, n_path) -> None:
    old = {n: None if cache[n] is None else cache[n].copy() for n in ("k", "v", "k_scale", "v_scale")}
    for r in range(len(base)):
        if not 0 <= n_path[r] <= path.shape[1] or base[r] < 0:
            continue
        for i in range(int(n_path[r])):
            if not 0 <= path[r, i] < 64:
                continue
            a, b = place(cache, r, int(base[r]) + int(path[r, i])), place(cache, r, int(base[r]) + i)
            if a is None or b is None:
                continue
            for n, x in old.items():
                if x is not None:
                    cache[n][b[0], :, b[1]] = x[a[0], :, a[1]]


def seen(j: int, n: int, base: int, tree_word) -> np.ndarray:
    """Boolean [base + n]: what row j of a request's n rows sees."""
    own = np.array([t <= j if tree_word is None else bool((int(tree_word) >> t) & 1) for t in range(n)], dtype=bool)
    return np.concatenate([np.ones(base, dtype=bool), own])


def attention(cache: dict, q, offsets, base, scale: float, tree=None, weights: bool = False):
    """out [N, q heads, D]; rows of no request stay NaN.  With weights also, for the tolerances, the sum over what a row
    sees of p |v| and p |score|, and of p times the size of the products behind a score."""
    N, Hq, D = q.shape
    heads = cache["k"].shape[1]
    out = np.full((N, Hq, D), np.nan)
    mag, size = np.zeros((N, Hq, D)), np.zeros((N, Hq))
    for r in range(len(base)):
        lo, hi = int(offsets[r]), int(offsets[r + 1])
        if hi == lo:
            continue
        n, b = hi - lo, int(base[r])
        k, v = rows(cache, "k", r, range(b + n)), rows(cache, "v", r, range(b + n))
        here = np.array([place(cache, r, t) is not None for t in range(b + n)], dtype=bool)
        for j in range(n):
            at = np.flatnonzero(seen(j, n, b, None if tree is None else tree[lo + j]) & here)
            for h in range(Hq):
                if at.size == 0:
                    out[lo + j, h] = 0.0
                    continue
                kk, vv = k[at, h // (Hq // heads)], v[at, h // (Hq // heads)]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = scale * (kk @ q[lo + j, h])
                    e = np.exp(s - s.max())
                    p = e / e.sum()
                    out[lo + j, h] = p @ vv
                    if weights:
                        mag[lo + j, h] = p @ np.abs(vv)
                        size[lo + j, h] = (abs(scale) * (np.abs(kk) @ np.abs(q[lo + j, h]))).max()
    return (out, mag, size) if weights else out
