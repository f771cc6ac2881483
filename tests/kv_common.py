"""A paged cache on the GPU and the same one in NumPy, for the tests of the cache operators and the attention."""
from __future__ import annotations

import numpy as np
import torch

from draft_sampling_lossless_markov_gb300 import torch_api as T
from oracle.vocab import e4m3_decode

E4M3, BF16, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32


def np64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def bits(t):
    """The bytes of a tensor, to compare them whole."""
    return t.contiguous().view(torch.uint8)


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def values(t):
    """What a pool's elements stand for, in fp64."""
    return e4m3_decode(t.contiguous().view(torch.uint8).cpu().numpy()) if t.dtype == E4M3 else np64(t)


def make_cache(g, dtype, tokens, heads, D, page, spare=2, fill="normal") -> T.KvCache:
    """Room for tokens[r] of request r in pages dealt out at random; entries of the table past them are out of range.
    fill "nan": every element and scale that holds no token is NaN."""
    per = [-(-t // page) for t in tokens]
    n_pages = sum(per) + spare
    order = torch.randperm(n_pages, generator=g, device="cuda").tolist()
    table = np.full((max(1, len(per)), max(1, max(per, default=1))), -7, dtype=np.int64)
    table[:, 1::2] = 2 ** 30
    for r, n in enumerate(per):
        for i in range(n):
            table[r, i] = order.pop()
    table = table[:len(per)]
    shape = (n_pages, heads, page, D)
    k, v = (torch.randn(shape, generator=g, device="cuda") for _ in range(2))
    used = torch.zeros((n_pages, 1, page, 1), dtype=torch.bool, device="cuda")
    for r, t in enumerate(tokens):
        for i in range(per[r]):
            used[int(table[r, i]), 0, :min(page, t - i * page)] = True
    if fill == "nan":
        k, v = (torch.where(used, x, torch.full_like(x, float("nan"))) for x in (k, v))
    if dtype == BF16:
        return T.KvCache(k.to(BF16), v.to(BF16), i32(table))
    ks, vs = (torch.exp(0.7 * torch.randn(shape[:3], generator=g, device="cuda")) / 100 for _ in range(2))
    if fill == "nan":
        ks, vs = (torch.where(used[..., 0], x, torch.full_like(x, float("nan"))) for x in (ks, vs))
    return T.KvCache((k * 100).clamp(-448, 448).to(E4M3), (v * 100).clamp(-448, 448).to(E4M3), i32(table), ks, vs)


def as_numpy(c: T.KvCache) -> dict:
    scale = lambda t: None if t is None else np64(t)  # noqa: E731
    return dict(k=values(c.k), v=values(c.v), k_scale=scale(c.k_scale), v_scale=scale(c.v_scale), table=c.table.cpu().numpy())


def clone(c: T.KvCache) -> T.KvCache:
    own = lambda t: None if t is None else t.view(torch.uint8).clone().view(t.dtype)  # noqa: E731
    return T.KvCache(own(c.k), own(c.v), c.table.clone(), own(c.k_scale), own(c.v_scale))


def parts(c: T.KvCache) -> list:
    return [t for t in (c.k, c.v, c.k_scale, c.v_scale) if t is not None]
