"""GPU parity of tree_attention against the fp64 oracle.

Tolerances, derived before the first run.  A score is a sum of at most 2 D products of e4m3 codes (bf16 values: D), exact
in fp32, with fp32 additions; q is exact or within 2^-18 of its row's largest element.  With size = |scale| sum |q| |k|
(the oracle's, the largest over a row's tokens) a score is within 2^-17 size, its exponent's arithmetic adds 2^-20 (1 +
size), and the weights, normalised, carry twice that.  A weight enters the sum over v within 2^-8 of it; weights far below
the largest within 2^-23 of the largest.  The result is rounded to bf16, 2^-8.  With mag = sum p |v|:
    |got - want| <= mag (2^-8 + 2^-15 size + 2^-18) + 2^-8 |want| + 2^-20 max |v|.
These errors have no common sign, so over all elements they add up to far less: the output's rounding alone is 0.0017 of
the norm, rounded weights add at most as much again: 0.004 is allowed.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from draft_sampling_lossless_markov_gb300 import capi
from draft_sampling_lossless_markov_gb300 import torch_api as T
from gpu_common import check_no_error, require_gpu
from kv_common import BF16, E4M3, as_numpy, bits, i32, make_cache, np64
from oracle import kv_cache as O

pytestmark = pytest.mark.gpu

NORM = 0.004


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def random_tree(rng, counts):
    """A word a row: itself and its ancestors, parents among the nodes before."""
    words = []
    for n in counts:
        mine = []
        for j in range(n):
            mine.append((1 << j) | (mine[rng.integers(0, j)] if j else 0))
        words += mine
    return np.array(words, dtype=np.uint64)


def i64(words):
    return torch.from_numpy(np.asarray(words, dtype=np.uint64).view(np.int64).copy()).cuda()


def setup(seed, dtype, base, counts, heads, group, D, page, tree=False, fill="nan", sharp=2.0):
    g = gen(seed)
    rng = np.random.default_rng(seed)
    c = make_cache(g, dtype, [b + n for b, n in zip(base, counts)], heads, D, page, fill=fill)
    N = int(sum(counts))
    qkv = (sharp * torch.randn((N, (heads * group + 2 * heads) * D), generator=g, device="cuda")).to(BF16)
    q = qkv[:, :heads * group * D].view(N, heads * group, D)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    words = random_tree(rng, counts) if tree else None
    return c, q, offsets, words


def call(c, q, offsets, base, words, max_tree, **kw):
    ws = kw.pop("ws", None) or T.tree_attention_workspace(c.n_req, max_tree, q.shape[1], c.n_kv_heads, c.head_dim)
    out = T.tree_attention(ws, c, q, i32(offsets), i32(base), max_tree, tree=None if words is None else i64(words), **kw)
    check_no_error(ws)
    return out


def check(c, q, offsets, base, words, out, scale=None, rows=None):
    ref = as_numpy(c)
    scale = c.head_dim ** -0.5 if scale is None else scale
    want, mag, size = O.attention(ref, np64(q), offsets, base, scale, words, weights=True)
    got = np64(out)
    if rows is not None:
        got, want, mag, size = got[rows], want[rows], mag[rows], size[rows]
    nan = np.isnan(want)
    np.testing.assert_array_equal(np.isnan(got), nan)
    vmax = np.nanmax(np.abs(ref["v"] * (1 if ref["v_scale"] is None else ref["v_scale"][..., None])))
    with np.errstate(invalid="ignore"):
        slack = mag * (2.0 ** -8 + 2.0 ** -15 * size[..., None] + 2.0 ** -18) + 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * vmax
    off = np.abs(got - want)[~nan]
    assert (off <= slack[~nan]).all(), (off / slack[~nan]).max()
    norm = np.linalg.norm(want[~nan])
    if norm > 0:
        assert np.linalg.norm(off) / norm < NORM, np.linalg.norm(off) / norm


CASES = [  # base, rows, kv heads, group, D, page, tree
    ([0], [1], 1, 1, 64, 16, False), ([1], [1], 2, 4, 128, 16, False), ([300], [1], 8, 4, 128, 64, False),
    ([127, 128, 129, 126], [1, 1, 1, 1], 2, 2, 128, 16, False), ([0, 5, 0], [64, 1, 3], 1, 2, 128, 32, True),
    ([100, 0, 250, 31], [8, 8, 8, 8], 4, 4, 128, 64, False), ([17, 640, 0, 3], [0, 5, 0, 13], 2, 7, 64, 16, True),
    ([700], [16], 2, 4, 128, 256, True), ([1000], [3], 1, 16, 64, 1024, True), ([63, 64, 65], [64, 63, 62], 1, 1, 64, 128, True),
    ([200, 90], [33, 20], 2, 8, 128, 16, True), ([5] * 40, [1, 2, 0, 3] * 10, 2, 3, 64, 16, True),
    ([120], [20], 1, 5, 128, 32, False), ([2500], [2], 3, 1, 128, 64, False), ([511, 1], [64, 64], 1, 4, 64, 64, True),
]


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", "")[:60])
def test_parity(case, dtype):
    base, counts, heads, group, D, page, tree = case
    c, q, offsets, words = setup(sum(base) + page, dtype, base, counts, heads, group, D, page, tree)
    out = call(c, q, offsets, base, words, max(1, max(counts)))
    check(c, q, offsets, base, words, out)


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("max_tree", [5, 16, 40, 64])
def test_fewer_rows_than_the_most_there_may_be(max_tree, dtype):
    base, counts = [140, 9, 0], [5, 1, 3]
    c, q, offsets, words = setup(3, dtype, base, counts, 2, 4, 128, 32, True)
    check(c, q, offsets, base, words, call(c, q, offsets, base, words, max_tree))


@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_strided_rows_and_untouched_places(dtype):
    base, counts = [33, 260], [6, 3]
    c, q, offsets, words = setup(4, dtype, base, counts, 2, 3, 64, 16, True)
    wide = torch.full((15, 6 * 64 + 8), 3.0, dtype=BF16, device="cuda")
    q15 = torch.zeros((15, 6, 64), dtype=BF16, device="cuda")
    q15[:9] = q
    out = wide[:, :6 * 64].view(15, 6, 64)
    call(c, q15, offsets, base, np.concatenate([words, np.zeros(6, dtype=np.uint64)]), 7, out=out)
    check(c, q, offsets, base, words, out[:9])
    assert (out[9:] == 3.0).all() and (wide[:, 6 * 64:] == 3.0).all()


@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_rows_that_see_nothing(dtype):
    base, counts = [0, 40, 0], [4, 2, 3]
    c, q, offsets, words = setup(5, dtype, base, counts, 2, 2, 64, 16, True)
    words[1] = words[3] = words[4] = words[6] = 0
    words[2] |= np.uint64(1 << 40)  # a bit past the request's rows
    out = call(c, q, offsets, base, words, 4)
    check(c, q, offsets, base, np.array([int(w) & 15 for w in words]), out)
    assert (out[[1, 3, 6]] == 0).all() and (out[4] != 0).any()


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("base,page", [(0, 16), (100, 16), (250, 64)])
def test_nan_and_infinity_in_hidden_rows(base, page, dtype):
    """Drafted rows hold NaN or infinities: only the rows that see them are touched."""
    counts, heads, D = [6], 2, 64
    c, q, offsets, _ = setup(6, dtype, [base], counts, heads, 2, D, page, True)
    words = np.array([1, 3, 0b101, 0b1001, 0b10011, 0b100101], dtype=np.uint64)

    def at(t):
        p = base + t
        return int(c.table[0, p // page]), p % page

    bad = float("nan")
    for t, name in ((1, "v"), (2, "k"), (3, "v")):
        a, b = at(t)
        x = getattr(c, name)
        if dtype == E4M3:
            x.view(torch.uint8)[a, :, b, 7] = 0x7F
        else:
            x[a, :, b, 7] = bad if t < 3 else float("inf")
            if t == 3:
                x[a, 1, b, 9] = float("-inf")
    out = call(c, q, offsets, [base], words, 6)
    got = np64(out)
    # row 0 sees none of them; 1 and 4 see v of 1; 2 and 5 see k of 2; 3 sees v of 3
    np.testing.assert_array_equal(np.isnan(got[2]), True)
    np.testing.assert_array_equal(np.isnan(got[5]), True)
    for j in (1, 4):
        assert np.isnan(got[j, :, 7]).all() and np.isfinite(np.delete(got[j], 7, 1)).all()
    if dtype == E4M3:
        assert np.isnan(got[3, :, 7]).all() and np.isfinite(np.delete(got[3], 7, 1)).all()
    else:
        assert (got[3, :, 7] == np.inf).all() and (got[3, 2:, 9] == -np.inf).all() and np.isfinite(got[3, :2, 9]).all()
    clean, qc, oc, _ = setup(6, dtype, [base], counts, heads, 2, D, page, True)  # the same numbers without them
    want = O.attention(as_numpy(clean), np64(qc), oc, [base], D ** -0.5, words)
    for j, cols in ((0, slice(None)), (1, slice(8, None)), (3, slice(10, None)), (4, slice(0, 7))):
        assert np.linalg.norm(got[j, :, cols] - want[j, :, cols]) < NORM * np.linalg.norm(want[j])


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("what", ["k", "v", "q", "scale"])
def test_nan_in_sight(what, dtype):
    base, counts = [150], [2]
    c, q, offsets, _ = setup(7, dtype, base, counts, 2, 2, 64, 16)
    if what == "scale" and dtype == BF16:
        pytest.skip("a bf16 cache has no scales")
    q = q.clone()
    page, slot = int(c.table[0, 130 // 16]), 130 % 16
    if what == "q":
        q[1, 2, 3] = float("inf")
    elif what == "scale":
        c.v_scale[page, 1, slot] = float("nan")
    elif dtype == E4M3:
        getattr(c, what).view(torch.uint8)[page, 1, slot, 3] = 0xFF
    else:
        getattr(c, what)[page, 1, slot, 3] = float("nan")
    got = np64(call(c, q, offsets, base, None, 2))
    nan = np.zeros_like(got, dtype=bool)
    if what == "q":
        nan[1, 2] = True
    elif what == "v":
        nan[:, 2:, 3] = True
    else:
        nan[:, 2:] = True
    np.testing.assert_array_equal(np.isnan(got), nan)


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("order", ["rising", "falling", "sink", "late"])
def test_scores_far_apart(order, dtype):
    """A running maximum that keeps rising or never does, one token far above a long tail, and one at the end."""
    base, D, page = [1400], 64, 32
    c, q, offsets, _ = setup(8, dtype, base, [2], 1, 2, D, page, fill="normal", sharp=0.02)
    t = torch.arange(1402, device="cuda")
    want = {"rising": t / 20.0, "falling": -t / 20.0, "sink": torch.where(t == 0, 9.0, 0.0), "late": torch.where(t == 1390, 60.0, 0.0)}[order]
    q[..., 0] = 8.0  # the score is scale * 8 * k[0], and small others
    pages = c.table[0].long()
    col = torch.zeros((len(pages) * page,), device="cuda")
    col[:1402] = want * D ** 0.5 / 8.0
    if dtype == BF16:
        c.k[pages, 0, :, 0] = col.view(-1, page).to(BF16)
    else:
        s = c.k_scale[pages, 0]
        s = torch.where(col.view(-1, page) != 0, col.view(-1, page).abs() / 448, s / 100)
        c.k_scale[pages, 0] = s
        c.k[pages, 0, :, 0] = (col.view(-1, page) / s).clamp(-448, 448).to(E4M3)
    check(c, q, offsets, base, None, call(c, q, offsets, base, None, 2))


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scales(scale):
    base, counts = [300, 20], [4, 9]
    c, q, offsets, words = setup(9, E4M3, base, counts, 2, 4, 128, 16, True)
    check(c, q, offsets, base, words, call(c, q, offsets, base, words, 9, scale=scale), scale=scale)


def test_rows_of_zeros_and_of_very_different_scales():
    """Values of zero with the least scale, and scales from 2^-60 to 2^40 (a token far above sets its row's size)."""
    base, counts = [200], [3]
    c, q, offsets, _ = setup(10, E4M3, base, counts, 2, 2, 64, 16)
    c.v_scale[:] = torch.exp2(torch.randint(-60, 41, c.v_scale.shape, generator=gen(1), device="cuda").float())
    check(c, q, offsets, base, None, call(c, q, offsets, base, None, 3))
    c.v.view(torch.uint8)[:] = 0
    c.v_scale[:] = 2.0 ** -100 / 448
    assert (call(c, q, offsets, base, None, 3) == 0).all()
    c.v_scale[:] = 0.0  # a cache that was cleared by hand
    assert (call(c, q, offsets, base, None, 3) == 0).all()


def test_small_elements_of_q():
    """Elements of one q row 2^-30 .. 1 of the largest: those that score on their own still score."""
    base, counts = [260], [2]
    c, q, offsets, _ = setup(11, E4M3, base, counts, 1, 2, 128, 32)
    q = (q.float() * torch.exp2(-torch.arange(128, device="cuda") % 31.0)).to(BF16)
    check(c, q, offsets, base, None, call(c, q, offsets, base, None, 2))
    q = (q.float() * 2.0 ** -100).to(BF16)
    check(c, q, offsets, base, None, call(c, q, offsets, base, None, 2))
    check(c, q, offsets, base, None, call(c, q, offsets, base, None, 2, scale=2.0 ** 99), scale=2.0 ** 99)
    assert torch.isfinite(call(c, torch.zeros_like(q), offsets, base, None, 2)).all()


@pytest.mark.parametrize("bad", ["base", "rows", "order", "past N", "past the table"])
def test_requests_out_of_range_are_left_out_and_reported(bad):
    base, counts = [30, 50, 20], [3, 4, 2]
    c, q, offsets, _ = setup(12, E4M3, base, counts, 2, 2, 64, 16)
    offsets, max_tree, where = offsets.copy(), 4, 1
    want = call(c, q, offsets, base, None, 4)
    if bad == "base":
        base[1] = -1
    elif bad == "rows":
        max_tree = 3
    elif bad == "order":
        offsets[2] = offsets[1] - 1
        offsets[3], where = offsets[2] + 2, 1
    elif bad == "past N":
        offsets[2], offsets[3] = 11, 11
    else:
        base[1] = c.table.shape[1] * 16 - 3
    out = torch.full_like(q, 9.0)
    ws = T.tree_attention_workspace(3, 4, 4, 2, 64)
    T.tree_attention(ws, c, q, i32(offsets), i32(base), max_tree, out=out)
    code, detail = ws.read_error()  # the request after one that ends past N begins there
    assert code == capi.DSPARK_BAD_INPUT and (detail == where or (bad == "past N" and detail == 2))
    if bad != "order":
        assert (out[3:7] == 9.0).all()
        assert torch.equal(bits(out[:3]), bits(want[:3])) or np.linalg.norm(np64(out[:3] - want[:3])) < NORM * np.linalg.norm(np64(want[:3]))


@pytest.mark.parametrize("page_id", [-1, 10 ** 6])
@pytest.mark.parametrize("at", [0, 3, 8, 12])
@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_pages_out_of_range_are_not_seen(dtype, at, page_id):
    base, counts = [190, 20], [7, 2]
    c, q, offsets, words = setup(13, dtype, base, counts, 2, 2, 64, 16, True)
    c.table[0, at] = page_id
    ws = T.tree_attention_workspace(2, 7, 4, 2, 64)
    out = T.tree_attention(ws, c, q, i32(offsets), i32(base), 7, tree=i64(words))
    assert ws.read_error() == (capi.DSPARK_BAD_INPUT, 0)
    check(c, q, offsets, base, words, out)


def test_no_rows_and_no_requests():
    c, q, offsets, _ = setup(14, E4M3, [20, 30], [0, 0], 2, 2, 64, 16)
    out = torch.full((3, 4, 64), 2.0, dtype=BF16, device="cuda")
    q = torch.zeros_like(out)
    call(c, q, [0, 0, 0], [20, 30], None, 4, out=out)
    assert (out == 2.0).all()
    call(c, q[:0], [0, 0, 0], [20, 30], None, 4)


def test_shared_pages():
    """Requests that begin with the same text share its pages."""
    base, counts = [160, 160, 160], [2, 3, 1]
    c, q, offsets, words = setup(15, E4M3, base, counts, 2, 4, 128, 16, True)
    c.table[1, :10] = c.table[0, :10]
    c.table[2, :10] = c.table[0, :10]
    check(c, q, offsets, base, words, call(c, q, offsets, base, words, 3))


@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_equal_calls_give_equal_bits(dtype):
    base, counts = [3000, 10, 900, 0], [8, 8, 3, 8]
    c, q, offsets, words = setup(16, dtype, base, counts, 4, 4, 128, 64, True)
    first = call(c, q, offsets, base, words, 8)
    for _ in range(5):
        torch.empty(64 << 20, device="cuda").normal_()
        assert torch.equal(bits(first), bits(call(c, q, offsets, base, words, 8)))


def test_graph_with_lengths_that_change():
    """A captured call replayed as contexts grow, requests end and trees change."""
    heads, group, D, page = 2, 4, 128, 16
    c, q, offsets, words = setup(17, E4M3, [600, 500, 400], [8, 8, 8], heads, group, D, page, True, fill="normal")
    off, base, tree = i32(offsets), i32([0, 0, 0]), i64(words)
    ws = T.tree_attention_workspace(3, 8, heads * group, heads, D)
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        T.tree_attention(ws, c, q, off, base, 8, tree=tree, out=out)
    for b, n in (([0, 0, 0], [8, 8, 8]), ([600, 131, 5], [8, 0, 8]), ([10, 500, 399], [1, 8, 0]), ([600, 500, 400], [3, 2, 1])):
        o = np.concatenate([[0], np.cumsum(n)])
        w = random_tree(np.random.default_rng(sum(b)), n)
        off.copy_(i32(o)), base.copy_(i32(b))
        tree[:len(w)] = i64(w)
        q.normal_(generator=gen(sum(b)))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        check_no_error(ws)
        check(c, q[:o[-1]], o, b, w, out[:o[-1]])
        assert (out[o[-1]:] == 7.0).all()


def test_streams_at_once():
    """Calls on four streams, each with its own workspace, among other work."""
    made = [setup(20 + i, (E4M3, BF16)[i % 2], [400 * (i + 1), 77], [8, 5], 2, 4, 128, 32, True) for i in range(4)]
    want = [call(*m[:3], [400 * (i + 1), 77], m[3], 8) for i, m in enumerate(made)]
    ws = [T.tree_attention_workspace(2, 8, 8, 2, 128) for _ in range(4)]
    args = [(i32(m[2]), i32([400 * (i + 1), 77]), i64(m[3]), torch.zeros_like(m[1])) for i, m in enumerate(made)]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            off, base, tree, out = args[i]
            T.tree_attention(ws[i], made[i][0], made[i][1], off, base, 8, tree=tree, out=out, stream=s)
    torch.cuda.synchronize()
    for i in range(4):
        check_no_error(ws[i])
        assert torch.equal(bits(args[i][3]), bits(want[i]))


@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_step_by_step(dtype):
    """Two rounds of write, attend, keep a path: every kept row's output is that of decoding it alone, one token at a time."""
    heads, group, D, page, B = 2, 4, 64, 16, 3
    rng = np.random.default_rng(0)
    g = gen(30)
    base = np.array([40, 0, 130])
    c = make_cache(g, dtype, list(base + 64 + 64), heads, D, page)
    ws = T.tree_attention_workspace(B, 12, heads * group, heads, D)
    for _ in range(2):
        counts = rng.integers(2, 13, B)
        offsets = np.concatenate([[0], np.cumsum(counts)])
        words = random_tree(rng, counts)
        N = int(offsets[-1])
        q = (2 * torch.randn((N, heads * group, D), generator=g, device="cuda")).to(BF16)
        k, v = (torch.randn((N, heads, D), generator=g, device="cuda").to(BF16) for _ in range(2))
        req = np.repeat(np.arange(B), counts)
        pos = np.concatenate([np.arange(n) for n in counts])
        T.cache_write(c, k, v, i32(req), i32(pos), base=i32(base), ws=ws)
        out = T.tree_attention(ws, c, q, i32(offsets), i32(base), 12, tree=i64(words))
        check(c, q, offsets, base, words, out)
        # the path to a random leaf
        path, n_path = np.zeros((B, 12), dtype=np.int64), np.zeros(B, dtype=np.int64)
        for r in range(B):
            leaf = int(words[offsets[r] + rng.integers(0, counts[r])])
            nodes = [t for t in range(counts[r]) if leaf >> t & 1]
            path[r, :len(nodes)], n_path[r] = nodes, len(nodes)
        T.cache_move(c, i32(base), i32(path), i32(n_path), ws=ws)
        check_no_error(ws)
        for step in range(int(n_path.max())):  # the same rows, one at a time over the cache as it now is
            live = np.flatnonzero(n_path > step)
            rows = [int(offsets[r] + path[r, step]) for r in live]
            one = np.concatenate([[0], np.cumsum(n_path > step)])
            alone = T.tree_attention(ws, c, q[rows].contiguous(), i32(one), i32(base + np.where(n_path > step, step, 0)), 1)
            a, b = np64(alone), np64(out[rows])
            assert np.linalg.norm(a - b) < NORM * np.linalg.norm(b)
        base = base + n_path
    check_no_error(ws)


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("seed", range(12))
def test_drawn_shapes(seed, dtype):
    """Sizes, head layouts, pages and trees drawn at random, rows from none to the most."""
    rng = np.random.default_rng(100 + seed)
    B, D, page = int(rng.integers(1, 9)), int(rng.choice([64, 128])), 16 << int(rng.integers(0, 7))
    heads, group, most = int(rng.integers(1, 5)), int(rng.choice([1, 2, 3, 5, 8, 11])), int(rng.integers(1, 65))
    base = [int(x) for x in np.exp(rng.uniform(0, 7.5, B)) - 1]
    counts = [int(x) for x in rng.integers(0, most + 1, B)]
    counts[0] = most
    c, q, offsets, words = setup(200 + seed, dtype, base, counts, heads, group, D, page, bool(seed % 3))
    check(c, q, offsets, base, words, call(c, q, offsets, base, words, most))


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("group,rows,D", [(64, 3, 128), (100, 5, 64), (33, 64, 64), (1000, 1, 64)])
def test_many_query_heads_a_kv_head(group, rows, D, dtype):
    base, counts = [70, 0, 333], [rows, 0, max(1, rows // 2)]
    c, q, offsets, words = setup(group, dtype, base, counts, 1, group, D, 64, True)
    check(c, q, offsets, base, words, call(c, q, offsets, base, words, rows))


@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_more_requests_than_threads(dtype):
    """Requests of every kind, without rows, without a context and without both, more than a CTA has threads."""
    rng = np.random.default_rng(4)
    B = 1500
    base = [int(x) for x in rng.integers(0, 40, B) * (rng.random(B) < 0.7)]
    counts = [int(x) for x in rng.integers(0, 4, B)]
    c, q, offsets, words = setup(31, dtype, base, counts, 2, 2, 64, 16, True)
    check(c, q, offsets, base, words, call(c, q, offsets, base, words, 3))


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("rows,group,D,page", [(1, 2, 128, 64), (9, 3, 128, 512), (5, 8, 64, 16), (30, 2, 128, 32), (64, 4, 64, 1024)])
def test_one_context_over_many_ctas(rows, group, D, page, dtype):
    base, counts = [30011], [rows]
    c, q, offsets, words = setup(32, dtype, base, counts, 1, group, D, page, True)
    check(c, q, offsets, base, words, call(c, q, offsets, base, words, rows))


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("rows,group,D", [(4, 4, 128), (8, 4, 128), (16, 4, 128), (16, 4, 64), (12, 12, 128)])
def test_many_tiles_a_cta_from_memory(rows, group, D, dtype):
    """Long runs of tiles whose loads are late: contexts out of cache, more tiles than stages for every CTA."""
    rng = np.random.default_rng(6)
    B, heads = 20, 8
    base = [int(x) for x in rng.integers(0, 3500, B)]
    c, q, offsets, words = setup(33, dtype, base, [rows] * B, heads, group, D, 128, True, fill="normal")
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    ws = T.tree_attention_workspace(B, rows, heads * group, heads, D)
    outs = []
    for i in range(4):
        flush.fill_(i)
        outs.append(call(c, q, offsets, base, words, rows, ws=ws))
    check(c, q, offsets, base, words, outs[0])
    for out in outs[1:]:
        assert torch.equal(bits(out), bits(outs[0]))


def test_two_graphs_share_a_workspace():
    """Captured calls of different sizes with one workspace, replayed in turn without a wait between them."""
    made = [setup(40, E4M3, [900, 3], [8, 5], 2, 4, 128, 32, True), setup(41, BF16, [50] * 30, [2] * 30, 2, 2, 64, 16, True)]
    bases, most = [[900, 3], [50] * 30], [8, 2]
    want = [call(*m[:3], b, m[3], n) for m, b, n in zip(made, bases, most)]
    ws = T.tree_attention_workspace(30, 8, 8, 2, 128)
    args = [(i32(m[2]), i32(b), i64(m[3]), torch.zeros_like(m[1])) for m, b in zip(made, bases)]
    graphs = []
    for m, (off, base, tree, out), n in zip(made, args, most):
        graphs.append(torch.cuda.CUDAGraph())
        torch.cuda.synchronize()
        with torch.cuda.graph(graphs[-1]):
            T.tree_attention(ws, m[0], m[1], off, base, n, tree=tree, out=out)
    for _ in range(20):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    check_no_error(ws)
    for (_, _, _, out), w in zip(args, want):
        assert torch.equal(bits(out), bits(w))


@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_calls_that_follow_each_other(dtype):
    """Steps of write, attend, keep a path, read back, enqueued as a whole: the bits of the same steps with a wait after
    every call."""
    B, rows, heads, group, D, steps = 5, 8, 2, 4, 128, 6
    rng = np.random.default_rng(5)
    start = make_cache(gen(50), dtype, [300, 0, 20, 90, 1000], heads, D, 16)
    pages = torch.zeros((B, 80), dtype=torch.int32)  # room for all the steps
    n = start.k.shape[0]
    k, v = (torch.cat([t.view(torch.uint8), torch.zeros((B * 80, *t.view(torch.uint8).shape[1:]), dtype=torch.uint8, device="cuda")])
            .view(t.dtype) for t in (start.k, start.v))
    scales = [] if dtype == BF16 else [torch.cat([t, torch.zeros((B * 80, *t.shape[1:]), device="cuda")])
                                       for t in (start.k_scale, start.v_scale)]
    pages[:] = n + torch.randperm(B * 80, generator=torch.Generator().manual_seed(1)).view(B, 80)
    old = start.table.cpu()
    for r, tokens in enumerate((300, 0, 20, 90, 1000)):
        m = -(-tokens // 16)
        pages[r, :m] = old[r, :m]
    data = [dict(k=torch.randn((B * rows, heads, D), generator=gen(60 + i), device="cuda").to(BF16),
                 v=torch.randn((B * rows, heads, D), generator=gen(70 + i), device="cuda"),
                 q=torch.randn((B * rows, heads * group, D), generator=gen(80 + i), device="cuda").to(BF16),
                 tree=i64(random_tree(rng, [rows] * B)), path=i32(np.sort(rng.integers(0, rows, (B, 4)), 1)),
                 n_path=i32(rng.integers(0, 5, B))) for i in range(steps)]
    req, pos, off = i32(np.repeat(np.arange(B), rows)), i32(np.tile(np.arange(rows), B)), i32(np.arange(B + 1) * rows)

    def run(wait):
        c = T.KvCache(k.view(torch.uint8).clone().view(k.dtype), v.view(torch.uint8).clone().view(k.dtype), pages.cuda(),
                      *(t.clone() for t in scales))
        ws = T.tree_attention_workspace(B, rows, heads * group, heads, D)
        base, outs = i32([300, 0, 20, 90, 1000]), []
        torch.cuda.synchronize()
        for d in data:
            for f in (lambda: T.cache_write(c, d["k"], d["v"].to(BF16), req, pos, base=base, ws=ws),
                      lambda: outs.append(T.tree_attention(ws, c, d["q"], off, base, rows, tree=d["tree"])),
                      lambda: T.cache_move(c, base, d["path"], d["n_path"], ws=ws),
                      lambda: outs.extend(T.cache_read(c, req, pos, base=base, ws=ws)), lambda: base.add_(d["n_path"])):
                f()
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        check_no_error(ws)
        return outs + [c.k.view(torch.uint8), c.v.view(torch.uint8)]

    for a, b in zip(run(False), run(True)):
        assert torch.equal(bits(a), bits(b))


FIRST_CALLS = """
import torch
from draft_sampling_lossless_markov_gb300 import torch_api as T
i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
g = torch.Generator(device="cuda").manual_seed(1)
for dt in (torch.bfloat16, torch.float8_e4m3fn):
    for D in (64, 128):
        for rows, heads in ((1, 4), (8, 8), (30, 4), (64, 16)):
            table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
            c = T.KvCache.create(40, 16, 2, D, table, dtype=dt)
            k, v = (torch.randn((2 * rows, 2, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
            q = torch.randn((2 * rows, heads, D), generator=g, device="cuda").to(torch.bfloat16)
            req, pos = torch.arange(2 * rows, device="cuda").int() // rows, torch.arange(2 * rows, device="cuda").int() % rows
            off, base, path, n_path = i32(0, rows, 2 * rows), i32(0, 200), i32(0, 0).view(2, 1), i32(1, 1)
            ws = T.tree_attention_workspace(2, rows, heads, 2, D)
            out, back = torch.zeros_like(q), (torch.zeros_like(k), torch.zeros_like(v))

            def call():
                T.cache_write(c, k, v, req, pos, base=base, ws=ws)
                T.tree_attention(ws, c, q, off, base, rows, out=out)
                T.cache_read(c, req, pos, base=base, out=back, ws=ws)
                T.cache_move(c, base, path, n_path, ws=ws)

            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                call()
            graph.replay()
            first = [t.clone() for t in (out, *back)]
            for t in (out, *back):
                t.zero_()
            call()
            torch.cuda.synchronize()
            assert ws.read_error()[0] == 0
            for a, b in zip(first, (out, *back)):
                assert a.abs().max() > 0 and torch.equal(a, b)
print("done")
"""


def test_first_calls_under_capture():
    """A process whose first call of each form is the one a stream capture records."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("done\n"), r.stdout + r.stderr


@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_offsets_past_32_bits(dtype):
    """A pool of more than 2^32 bytes, the request's pages at its end."""
    heads, D, page = 8, 128, 128
    n_pages = (1 << 32) // (heads * D * page) + 300
    k = torch.zeros((n_pages, heads, page, D), dtype=torch.uint8 if dtype == E4M3 else BF16, device="cuda")
    v = torch.zeros_like(k)
    scales = [torch.ones((n_pages, heads, page), device="cuda") for _ in range(2)] if dtype == E4M3 else []
    if dtype == E4M3:
        k, v = k.view(E4M3), v.view(E4M3)
    pages = [n_pages - 1, 0, n_pages - 200]
    c = T.KvCache(k, v, i32([pages]), *scales)
    g = gen(40)
    rows = [torch.randn((300, heads, D), generator=g, device="cuda").to(BF16) for _ in range(2)]
    ws = T.tree_attention_workspace(1, 3, heads * 2, heads, D)
    T.cache_write(c, *rows, i32(np.zeros(300)), i32(np.arange(300)), ws=ws)
    q = (2 * torch.randn((3, heads * 2, D), generator=g, device="cuda")).to(BF16)
    out = T.tree_attention(ws, c, q, i32([0, 3]), i32([297]), 3)
    check_no_error(ws)
    near = [t[pages] for t in ((k.view(torch.uint8), v.view(torch.uint8)) if dtype == E4M3 else (k, v))]
    small = T.KvCache(*(t.view(k.dtype) for t in near), i32([[0, 1, 2]]), *(s[pages].contiguous() for s in scales))
    check(small, q, [0, 3], [297], None, out)
    back = T.cache_read(c, i32(np.zeros(300)), i32(np.arange(300)), ws=ws)
    same = T.cache_read(small, i32(np.zeros(300)), i32(np.arange(300)), ws=ws)
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(back, same)) and float(back[0].float().abs().sum()) > 0
    T.cache_move(c, i32([200]), i32([[40, 60]]), i32([2]), ws=ws)
    T.cache_move(small, i32([200]), i32([[40, 60]]), i32([2]), ws=ws)
    check_no_error(ws)
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(T.cache_read(c, i32([0]), i32([201])), T.cache_read(small, i32([0]), i32([201]))))
