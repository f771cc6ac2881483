"""The vocabulary projection and the answers around verify, in fp64 — test infrastructure only.

* e4m3 quantisation with one scale for each block of 128 columns (and 1 or 128 rows);
* the product of two such matrices;
* log probability and rank of a given token, entropy, top alternatives, and their gradient.

Every function takes NumPy arrays; codes are uint8 e4m3 bit patterns.
"""
import numpy as np

BLOCK = 128
AMAX_MIN = 2.0 ** -100


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 e4m3 codes (1 sign, 4 exponent bits with bias 7, 3 mantissa bits;
    exponent 15 with mantissa 7 is NaN, there is no infinity)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


_VALUES = e4m3_values()


def e4m3_decode(codes: np.ndarray) -> np.ndarray:
    return _VALUES[codes]


def e4m3_round(x: np.ndarray) -> np.ndarray:
    """The e4m3 value nearest to x, ties to the even mantissa, at most 448 in magnitude."""
    x = np.asarray(x, np.float64)
    pos = _VALUES[:127]  # 0 .. 448 ascending; even codes have an even mantissa
    a = np.minimum(np.abs(x), 448.0)
    hi = np.minimum(np.searchsorted(pos, a, side="left"), 126)
    lo = np.maximum(hi - 1, 0)
    up, down = pos[hi] - a, a - pos[lo]
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0)) | (hi == 0)
    return np.copysign(np.where(take_hi, pos[hi], pos[lo]), x)


def quant(x: np.ndarray, block_rows: int):
    """(x * 448 / amax of its block before rounding to e4m3, scale [row blocks, column blocks])."""
    x = np.asarray(x, np.float64)
    M, K = x.shape
    rb, kb = -(-M // block_rows), -(-K // BLOCK)
    scaled, scale = np.empty((M, K)), np.empty((rb, kb))
    for i in range(rb):
        for b in range(kb):
            at = np.s_[i * block_rows:(i + 1) * block_rows, b * BLOCK:(b + 1) * BLOCK]
            blk = np.abs(x[at])
            amax = max(blk[np.isfinite(blk)].max(initial=0.0), AMAX_MIN)
            scale[i, b] = amax / 448.0
            with np.errstate(invalid="ignore"):
                scaled[at] = np.where(np.isfinite(x[at]), x[at], np.nan) * (448.0 / amax)
    return scaled, scale


def dequant(codes: np.ndarray, scale: np.ndarray, block_rows: int) -> np.ndarray:
    M, K = codes.shape
    return e4m3_decode(codes) * scale[np.arange(M) // block_rows][:, np.arange(K) // BLOCK]


def matmul(a, a_scale, w, w_scale):
    """(product, sum of the magnitudes of its terms)."""
    x, y = dequant(a, np.float64(a_scale), 1), dequant(w, np.float64(w_scale), BLOCK)
    return x @ y.T, np.abs(x) @ np.abs(y).T


def candidates(logits: np.ndarray, mask=None) -> np.ndarray:
    """Boolean [N, V]: not masked and above -inf (a NaN is a candidate)."""
    ok = ~np.isneginf(logits)
    if mask is not None:
        v = np.arange(logits.shape[1])
        ok &= ((mask.astype(np.uint32)[:, v >> 5] >> (v & 31).astype(np.uint32)) & 1).astype(bool)
    return ok


def temperature(T):
    T = np.asarray(T, np.float64)
    return np.where(np.isfinite(T) & (T > 0), T, 1.0)


def token_logprobs(logits, tokens, temp, top: int, mask=None) -> dict:
    """Row by row; logits fp64 [N, V], tokens [N] (-1: none), temp [N]."""
    N, V = logits.shape
    ok = candidates(logits, mask)
    T = temperature(temp)
    out = dict(logprob=np.zeros(N), entropy=np.zeros(N), rank=np.full(N, -1), row_stat=np.zeros((N, 2)),
               top_id=np.full((N, top), -1), top_logprob=np.full((N, top), -np.inf))
    for i in range(N):
        ids = np.flatnonzero(ok[i])
        x, tok = logits[i, ids], int(tokens[i])
        if ids.size == 0:
            out["logprob"][i] = -np.inf if tok >= 0 else 0.0
            out["row_stat"][i] = -np.inf, 0.0
            continue
        if np.isnan(x).any() or np.isposinf(x).any():
            out["logprob"][i] = np.nan if tok >= 0 else 0.0
            out["entropy"][i] = out["row_stat"][i, 1] = np.nan
            out["top_logprob"][i] = np.nan
            out["row_stat"][i, 0] = np.nan
            continue
        y = (x - x.max()) / T[i]
        S = np.exp(y).sum()
        logp = y - np.log(S)
        p = np.exp(logp)
        out["row_stat"][i] = x.max(), S
        out["entropy"][i] = -(p[p > 0] * logp[p > 0]).sum()
        order = np.lexsort((ids, -x))
        k = min(top, ids.size)
        out["top_id"][i, :k], out["top_logprob"][i, :k] = ids[order[:k]], logp[order[:k]]
        if tok >= 0:
            at = np.flatnonzero(ids == tok)
            out["logprob"][i] = logp[at[0]] if at.size else -np.inf
            if at.size:
                out["rank"][i] = int(np.flatnonzero(order == at[0])[0])
    return out


def _log_softmax(x, T):
    y = (x - x.max()) / T
    return y - np.log(np.exp(y).sum())


def loss(logits, tokens, temp, top_id, g_logprob, g_entropy, g_top, mask=None) -> np.ndarray:
    """[N]: the weighted sum of a row's outputs whose gradient token_logprobs_grad is, top_id held fixed;
    terms without a candidate are left out."""
    N = logits.shape[0]
    ok, T, out = candidates(logits, mask), temperature(temp), np.zeros(N)
    for i in range(N):
        ids = np.flatnonzero(ok[i])
        if ids.size == 0:
            continue
        logp = dict(zip(ids, _log_softmax(logits[i, ids], T[i])))
        lp = np.array(list(logp.values()))
        out[i] = g_entropy[i] * -(np.exp(lp) * lp).sum() + g_logprob[i] * logp.get(int(tokens[i]), 0.0)
        for g, v in zip(g_top[i], top_id[i]):
            out[i] += g * logp.get(int(v), 0.0)
    return out


def token_logprobs_grad(logits, tokens, temp, top_id, g_logprob, g_entropy, g_top, mask=None) -> np.ndarray:
    N, V = logits.shape
    ok, T, d = candidates(logits, mask), temperature(temp), np.zeros((N, V))
    for i in range(N):
        ids = np.flatnonzero(ok[i])
        if ids.size == 0:
            continue
        logp = _log_softmax(logits[i, ids], T[i])
        p = np.exp(logp)
        H = -(p * logp).sum()
        row = -g_entropy[i] * p * (logp + H)
        for g, v in [(g_logprob[i], int(tokens[i]))] + list(zip(g_top[i], top_id[i])):
            at = np.flatnonzero(ids == v)
            if at.size:
                row -= g * p
                row[at[0]] += g
        d[i, ids] = row / T[i]
    return d
