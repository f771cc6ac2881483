"""GPU parity of cache_write, cache_read and cache_move against the fp64 oracle.

Codes are those of the exact quotient, so they are equal where the quotient is not within 2^-22 of a tie between two
codes, and one of the two there (the oracle's quotient is rounded in fp64); scales are one fp32 division (2^-24).
Reads are one fp32 product (2^-24) and one rounding to bf16 (2^-8); of a bf16 cache they are exact.  Moves copy bytes.
"""
import numpy as np
import pytest
import torch

from draft_sampling_lossless_markov_gb300 import capi
from draft_sampling_lossless_markov_gb300 import torch_api as T
from gpu_common import check_no_error, require_gpu
from kv_common import BF16, E4M3, F32, as_numpy, bits, clone, i32, make_cache, np64, parts, values
from oracle import kv_cache as O
from oracle.vocab import e4m3_round

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def error_ws():
    return T.matmul_fp8_workspace(1, 1, 1)


CASES = [  # requests' lengths before and new rows, heads, D, page
    ([0], [1], 1, 64, 16), ([5, 0, 63, 64], [3, 17, 2, 1], 8, 128, 64), ([100, 15, 16], [40, 1, 90], 3, 64, 16),
    ([1000, 3], [5, 300], 5, 128, 256), ([7], [2050], 2, 128, 32), ([0, 9], [1, 2], 40, 64, 128), ([31], [6], 70, 128, 16),
]


def rows_of(counts, g):
    """Markers of every request's rows, in random order."""
    req = np.repeat(np.arange(len(counts)), counts)
    pos = np.concatenate([np.arange(n) for n in counts])
    order = torch.randperm(len(req), generator=g, device="cuda").cpu().numpy()
    return req[order], pos[order]


@pytest.mark.parametrize("cache_dtype", [E4M3, BF16])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_write(case, dtype, cache_dtype):
    base, counts, heads, D, page = case
    g = gen(1)
    c = make_cache(g, cache_dtype, [b + n for b, n in zip(base, counts)], heads, D, page)
    ref = as_numpy(c)
    req, pos = rows_of(counts, g)
    N = len(req)
    skip = np.zeros(N, dtype=bool)
    if N > 4:
        skip[::5] = True
    mark = np.where(skip, -1, req)
    wide = (torch.randn((N, 2 * heads * D + 16), generator=g, device="cuda") * torch.exp(2 * torch.randn(N, 1, generator=g, device="cuda"))).to(dtype)
    k, v = wide[:, :heads * D].view(N, heads, D), wide[:, heads * D:2 * heads * D].view(N, heads, D)
    v[0] = 0  # a row of zeros has the least scale
    ws = error_ws()
    T.cache_write(c, k, v, i32(mark), i32(pos), base=i32(base), ws=ws)
    check_no_error(ws)
    before = {n: None if x is None else x.copy() for n, x in ref.items()}
    assert O.write(ref, np64(k), np64(v), mark, pos, base, N, to_bf16=lambda x: np64(torch.tensor(x).to(BF16))) == []
    for n in ("k", "v"):
        got = values(getattr(c, n))
        if cache_dtype == BF16:
            np.testing.assert_array_equal(got, ref[n])
            continue
        np.testing.assert_allclose(np64(getattr(c, n + "_scale")), ref[n + "_scale"], rtol=2.0 ** -23)
        wrong = got != ref[n]
        assert wrong.mean() < 1e-3
        x = np64(k if n == "k" else v)
        for i in np.flatnonzero(~skip):  # a code beside the oracle's is on the other side of a tie
            at = O.place(ref, int(req[i]), base[req[i]] + int(pos[i]))
            q, _ = O.quant_row(x[i])
            lo, hi = e4m3_round(q * (1 - 2.0 ** -40)), e4m3_round(q * (1 + 2.0 ** -40))
            have = got[at[0], :, at[1]]
            assert ((np.minimum(lo, hi) <= have) & (have <= np.maximum(lo, hi))).all()
            before[n][at[0], :, at[1]] = have
        np.testing.assert_array_equal(got, before[n])  # nothing else was touched


def test_write_keeps_count_and_non_finite():
    g = gen(2)
    c = make_cache(g, E4M3, [40, 40], 2, 64, 16)
    old = clone(c)
    k = torch.randn((6, 2, 64), generator=g, device="cuda")
    v = k.clone()
    k[0, 0, 5], k[0, 1] = float("nan"), float("inf")
    ws = error_ws()
    T.cache_write(c, k, v, i32([0, 0, 1, 1, 1, 1]), i32([0, 1, 2, 3, 4, 5]), n_rows=i32([3]), ws=ws)
    check_no_error(ws)
    ref = as_numpy(old)
    O.write(ref, np64(k), np64(v), [0, 0, 1], [0, 1, 2], [0, 0], 3)
    for n in ("k", "v"):
        np.testing.assert_array_equal(values(getattr(c, n)), ref[n])
    at = O.place(ref, 0, 0)
    assert np.isnan(values(c.k)[at[0], 0, at[1], 5]) and np.isnan(values(c.k)[at[0], 1, at[1]]).all()
    for count in (0, -3):
        again = clone(c)
        T.cache_write(c, k, v, i32([0, 0, 1, 1, 1, 1]), i32([6, 7, 8, 9, 10, 11]), n_rows=i32([count]))
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(parts(c), parts(again)))
    T.cache_write(c, k[:0], v[:0], i32([]), i32([]))


@pytest.mark.parametrize("bad", ["request", "low request", "position", "negative position", "page", "large page"])
def test_rows_without_a_place_are_left_out_and_reported(bad):
    g = gen(3)
    c = make_cache(g, E4M3, [40, 40], 2, 64, 16)
    req, pos, base = [0, 1, 1], [0, 1, 2], [3, 4]
    if bad == "request":
        req[1] = 2
    elif bad == "low request":
        req[1] = -2
    elif bad == "position":
        pos[1] = 44
    elif bad == "negative position":
        pos[1] = -5
    else:
        pos[1] = 20  # page 1 of request 1
        c.table[1, 1] = -1 if bad == "page" else c.k.shape[0]
    old, ref = clone(c), as_numpy(c)
    k = torch.randn((3, 2, 64), generator=g, device="cuda")
    ws = error_ws()
    T.cache_write(c, k, k, i32(req), i32(pos), base=i32(base), ws=ws)
    assert ws.read_error() == (capi.DSPARK_BAD_INPUT, 1)
    assert O.write(ref, np64(k), np64(k), req, pos, base, 3) == [1]
    for n in ("k", "v"):
        np.testing.assert_array_equal(values(getattr(c, n)), ref[n])
    out = tuple(torch.full((3, 2, 64), 7.0, device="cuda") for _ in range(2))
    T.cache_read(c, i32(req), i32(pos), base=i32(base), out=out, ws=ws)
    assert ws.read_error() == (capi.DSPARK_BAD_INPUT, 1)
    assert (out[0][1] == 7).all() and (out[0][[0, 2]] != 7).all()
    T.cache_read(c, i32(req), i32(pos), base=i32(base), out=out)  # nothing to report to
    del old


@pytest.mark.parametrize("cache_dtype", [E4M3, BF16])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_read(case, dtype, cache_dtype):
    base, counts, heads, D, page = case
    g = gen(4)
    c = make_cache(g, cache_dtype, [b + n for b, n in zip(base, counts)], heads, D, page, fill="nan")
    req, pos = rows_of(counts, g)
    N = len(req)
    mark = np.where(np.arange(N) % 7 == 3, -1, req)
    wide = torch.full((N, 2 * heads * D + 8), 5.0, dtype=dtype, device="cuda")
    out = wide[:, :heads * D].view(N, heads, D), wide[:, heads * D:2 * heads * D].view(N, heads, D)
    ws = error_ws()
    n = N - N // 3
    T.cache_read(c, i32(mark), i32(pos), base=i32(base), n_rows=i32([n]), out=out, ws=ws)
    check_no_error(ws)
    live = (mark >= 0) & (np.arange(N) < n)
    ref = as_numpy(c)
    for name, t in zip(("k", "v"), out):
        got = np64(t)
        assert (got[~live] == 5.0).all()
        want = np.stack([O.rows(ref, name, int(r), [base[r] + p])[0] for r, p in zip(req, pos)])[live]
        if cache_dtype == BF16:
            np.testing.assert_array_equal(got[live], want)
        else:
            np.testing.assert_allclose(got[live], want, rtol=2.0 ** -23 + (2.0 ** -8 if dtype == BF16 else 0))
    assert (wide[:, 2 * heads * D:] == 5.0).all()


def test_what_is_written_is_read_back():
    g = gen(5)
    c = make_cache(g, E4M3, [300], 4, 128, 32)
    k, v = (torch.randn((300, 4, 128), generator=g, device="cuda") for _ in range(2))
    req, pos = i32(np.zeros(300)), i32(np.arange(300))
    T.cache_write(c, k, v, req, pos)
    for x, y in zip((k, v), T.cache_read(c, req, pos, dtype=F32)):
        # a code is off by at most half a step: 2^-4 of the value, 2^-10 of the scale's unit below the normal range
        slack = 2.0 ** -4 * x.abs() + 2.0 ** -10 * x.abs().amax(-1, keepdim=True) / 448 * 1.01
        assert ((x - y).abs() <= slack).all()
    twice = T.cache_read(c, i32([0, 0]), i32([9, 9]), dtype=F32)[0]
    assert torch.equal(twice[0], twice[1])


@pytest.mark.parametrize("cache_dtype", [E4M3, BF16])
@pytest.mark.parametrize("B,heads,D,page,cols", [(1, 1, 64, 16, 1), (5, 8, 128, 64, 8), (9, 3, 64, 16, 64), (33, 2, 128, 32, 5),
                                                 (4, 40, 128, 16, 64), (70, 1, 64, 16, 2), (3, 17, 64, 1024, 33)])
def test_move(B, heads, D, page, cols, cache_dtype):
    g = gen(6)
    rng = np.random.default_rng(B * cols)
    base = rng.integers(0, 90, B)
    c = make_cache(g, cache_dtype, list(base + 64), heads, D, page)
    path = np.stack([np.sort(rng.permutation(64)[:cols]) for _ in range(B)])
    path[::2, 0] = 0
    if B > 2:
        path[2] = rng.integers(0, 64, cols)  # any order, some twice
    n_path = rng.integers(0, cols + 1, B)
    n_path[0] = cols
    ref = as_numpy(c)
    O.move(ref, base, path, n_path)
    wide = torch.full((B, cols + 3), -9, dtype=torch.int32, device="cuda")
    wide[:, :cols] = i32(path)
    ws = error_ws()
    T.cache_move(c, i32(base), wide[:, :cols], i32(n_path), ws=ws)
    check_no_error(ws)
    for n in ("k", "v", "k_scale", "v_scale"):
        t = getattr(c, n)
        if t is not None:
            np.testing.assert_array_equal(np64(t) if n.endswith("scale") else values(t), ref[n])


@pytest.mark.parametrize("bad,where", [("count", 2), ("low count", 2), ("node", 1), ("negative node", 1), ("base", 0), ("page", 1),
                                       ("end", 0)])
def test_move_leaves_out_what_has_no_place(bad, where):
    g = gen(7)
    c = make_cache(g, E4M3, [80, 90, 100], 2, 64, 16)
    base, n_path = np.array([3, 20, 36]), np.array([4, 4, 4])
    path = np.tile(np.array([0, 3, 5, 9]), (3, 1))
    if bad == "count":
        n_path[2] = 5
    elif bad == "low count":
        n_path[2] = -1
    elif bad == "node":
        path[1, 2] = 64
    elif bad == "negative node":
        path[1, 2] = -1
    elif bad == "base":
        base[0] = -1
    elif bad == "page":
        c.table[1, (20 + 9) // 16] = -1
    else:
        base[0] = c.table.shape[1] * 16 - 6
        c.table[0] = c.table[0, 0]  # its last places exist
    ref = as_numpy(c)
    O.move(ref, base, path, n_path)
    ws = error_ws()
    T.cache_move(c, i32(base), i32(path), i32(n_path), ws=ws)
    assert ws.read_error() == (capi.DSPARK_BAD_INPUT, where)
    for n in ("k", "v"):
        np.testing.assert_array_equal(values(getattr(c, n)), ref[n])


def test_graph_and_streams():
    """A captured write, move and read of other contents than at capture, and calls on a stream of their own."""
    g = gen(8)
    side = torch.cuda.Stream()
    c = make_cache(g, E4M3, [100, 100], 8, 128, 16)
    k, v = (torch.randn((16, 8, 128), generator=g, device="cuda") for _ in range(2))
    req, pos, base = i32(np.repeat([0, 1], 8)), i32(np.tile(np.arange(8), 2)), i32([0, 30])
    path, n_path = i32([[0, 2, 5], [1, 3, 4]]), i32([3, 2])
    out = tuple(torch.zeros((16, 8, 128), dtype=BF16, device="cuda") for _ in range(2))

    def step():
        T.cache_write(c, k, v, req, pos, base=base)
        T.cache_move(c, base, path, n_path)
        T.cache_read(c, req, pos, base=base, out=out)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        k.normal_(generator=g), v.normal_(generator=g)
        base += 5
        path.copy_(torch.sort(torch.randint(0, 8, (2, 3), generator=g, device="cuda"), 1).values)
        ref = as_numpy(c)
        O.write(ref, np64(k), np64(v), req.cpu().numpy(), pos.cpu().numpy(), base.cpu().numpy(), 16)
        O.move(ref, base.cpu().numpy(), path.cpu().numpy(), n_path.cpu().numpy())
        if i < 2:
            graph.replay()
        else:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert (values(c.k) != ref["k"]).mean() < 1e-4
        want = np.stack([O.rows(as_numpy(c), "v", int(r), [int(base[int(r)]) + int(p)])[0] for r, p in zip(req, pos)])
        np.testing.assert_allclose(np64(out[1]), want, rtol=2.0 ** -8 + 2.0 ** -23)
