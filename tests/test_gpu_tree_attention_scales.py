"""GPU parity of tree_attention over e4m3 caches whose scales of v differ without bounds: rows of zeros as cache_write
makes them (scale 2^-100 / 448), cleared rows (scale 0, whatever their codes), the least and the largest normal scales.

Such a row's weight counts in the softmax's sum as any other's.  Tolerances, derived before the first run, are those of
test_gpu_tree_attention.py, with the part for small weights relative to the row's own largest product of a weight and a
scale of v instead of the cache's largest element: with n tokens, each within 2^-23 of that product times its code,
    |got - want| <= mag (2^-8 + 2^-15 size + 2^-18) + 2^-8 |want| + n 2^-23 448 max(p vs),
the last at most n 2^-14 max(p vs).  Weights that fp32 cannot hold beside the largest (below 2^-126 of it) do not count."""
import numpy as np
import pytest
import torch

import test_gpu_tree_attention as A
from draft_sampling_lossless_markov_gb300 import torch_api as T
from gpu_common import check_no_error, require_gpu
from kv_common import BF16, E4M3, as_numpy, i32, make_cache, np64

pytestmark = pytest.mark.gpu

ZERO_ROW = 2.0 ** -100 / 448


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def one_head(cache, r, n, scale):
    """(k, v, scales of v) of a request's first n tokens and of its only head, fp64."""
    page = cache["k"].shape[2]
    at = cache["table"][r, np.arange(n) // page], np.arange(n) % page
    k = cache["k"][at[0], 0, at[1]] * cache["k_scale"][at[0], 0, at[1]][:, None]
    vs = cache["v_scale"][at[0], 0, at[1]]
    return k, cache["v"][at[0], 0, at[1]] * vs[:, None], vs


def check_request(cache, r, q, got, base, scale):
    """A chain's rows q [rows, group, D] of one request over a cache of one head."""
    k, v, vs = one_head(cache, r, base + q.shape[0], scale)
    for j in range(q.shape[0]):
        n = base + j + 1
        s = scale * (q[j] @ k[:n].T)
        e = np.exp(s - s.max(-1, keepdims=True))
        p = e / e.sum(-1, keepdims=True)
        want, mag = p @ v[:n], p @ np.abs(v[:n])
        size = (abs(scale) * (np.abs(q[j]) @ np.abs(k[:n]).T)).max(-1)
        slack = mag * (2.0 ** -8 + 2.0 ** -15 * size[:, None] + 2.0 ** -18) + 2.0 ** -8 * np.abs(want) \
            + n * 2.0 ** -14 * (p * vs[:n]).max(-1)[:, None]
        off = np.abs(got[j] - want)
        assert (off <= slack).all(), (r, j, np.nanmax(off / slack), np.isnan(off).any())
        norm = np.linalg.norm(want)
        assert np.linalg.norm(off) <= A.NORM * norm, (r, j, np.linalg.norm(off) / norm)


def put_scales(c, r, first, count, value, clear=False):
    """The scales of v of a request's tokens first .. first + count - 1; `clear` takes their codes too."""
    page = c.k.shape[2]
    t = torch.arange(first, first + count, device="cuda")
    pages, slots = c.table[r].long()[t // page], t % page
    c.v_scale[pages, :, slots] = value
    if clear:
        c.v.view(torch.uint8)[pages, :, slots] = 0


FORMS = [(2, 2, 64), (1, 16, 128), (8, 4, 128), (4, 5, 64), (16, 4, 128), (9, 7, 64)]  # rows, heads, head size: 16, 32, 64 columns


@pytest.mark.parametrize("rows,group,D", FORMS)
@pytest.mark.parametrize("where", ["before", "between", "after", "all but the last"])
@pytest.mark.parametrize("value", [0.0, "zeros", ZERO_ROW, 2.0 ** -126, 2.0 ** -50])
def test_rows_of_zeros_among_others(value, where, rows, group, D):
    """Cleared rows and rows of zeros at one place of a context: one item and several, a tile and more."""
    clear = value in ("zeros", ZERO_ROW)
    value = 0.0 if value == "zeros" else value
    for base in (40, 300, 1000):
        c, q, offsets, _ = A.setup(base + rows, E4M3, [base], [rows], 1, group, D, 32, sharp=1.0)
        first, count = {"before": (0, base // 2), "between": (base // 3, base // 3), "after": (base // 2, base - base // 2),
                        "all but the last": (0, base + rows - 1)}[where]
        put_scales(c, 0, first, count, value, clear)
        got = np64(A.call(c, q, offsets, [base], None, rows))
        check_request(as_numpy(c), 0, np64(q), got, base, D ** -0.5)


@pytest.mark.parametrize("rows,group,D", FORMS)
@pytest.mark.parametrize("value", [0.0, ZERO_ROW])
def test_a_long_run_of_zeros(value, rows, group, D):
    """A context over many CTAs, several of which have nothing but rows of zeros."""
    base = 30000
    c, q, offsets, _ = A.setup(7, E4M3, [base], [rows], 1, group, D, 128, sharp=1.0)
    put_scales(c, 0, 0, base - 200, value, True)
    got = np64(A.call(c, q, offsets, [base], None, rows))
    check_request(as_numpy(c), 0, np64(q), got, base, D ** -0.5)


@pytest.mark.parametrize("rows,group,D", [(1, 16, 128), (8, 4, 128), (16, 4, 128)])
@pytest.mark.parametrize("value", [0.0, ZERO_ROW])
def test_items_of_one_cta(value, rows, group, D):
    """As many requests as there are CTAs, their contexts the same 12000 rows, all but the last 100 zeros: whole items."""
    base, B = 12000, 304
    c, q, _, _ = A.setup(8, E4M3, [base], [rows], 1, group, D, 128, fill="normal", sharp=1.0)
    put_scales(c, 0, 0, base - 100, value, True)
    many = T.KvCache(c.k, c.v, c.table.expand(B, -1).contiguous(), c.k_scale, c.v_scale)
    q = q.repeat(B, 1, 1)
    got = np64(A.call(many, q, np.arange(B + 1) * rows, [base] * B, None, rows))
    cache = as_numpy(c)
    for r in (0, 1, 151, 303):
        check_request(cache, 0, np64(q[:rows]), got[r * rows:(r + 1) * rows], base, D ** -0.5)


@pytest.mark.parametrize("rows,group,D", [(1, 16, 128), (8, 4, 128), (16, 4, 128)])
def test_zeros_that_score_far_higher(rows, group, D):
    """Rows of zeros whose scores are 20 above the others': they take nearly all of the weight."""
    base = 500
    c, q, offsets, _ = A.setup(9, E4M3, [base], [rows], 1, group, D, 16, sharp=0.05)
    put_scales(c, 0, 200, 150, ZERO_ROW, True)
    q[..., 0] = 4.0
    t = torch.arange(base, device="cuda")
    high = ((t >= 200) & (t < 350)).float() * 20 * D ** 0.5 / 4
    pages, slots = c.table[0].long()[t // 16], t % 16
    scale = torch.where(high > 0, high / 448, c.k_scale[pages, 0, slots])
    c.k_scale[pages, 0, slots] = scale
    codes = c.k[pages, 0, slots].float()
    codes[:, 0] = high / scale
    codes[high > 0, 1:] = 0
    c.k.view(torch.uint8)[pages, 0, slots] = codes.clamp(-448, 448).to(E4M3).view(torch.uint8)
    got = np64(A.call(c, q, offsets, [base], None, rows))
    check_request(as_numpy(c), 0, np64(q), got, base, D ** -0.5)


@pytest.mark.parametrize("rows,group,D", FORMS)
@pytest.mark.parametrize("small,large", [(0.0, 2.0 ** 100), (2.0 ** -126, 2.0 ** 119), (ZERO_ROW, 2.0 ** 30), (2.0 ** -126, 2.0 ** -126),
                                         (2.0 ** 119, 2.0 ** 119), (2.0 ** -60, 1.0)])
def test_the_least_and_the_largest_scales(small, large, rows, group, D):
    base = 700
    c, q, offsets, _ = A.setup(10, E4M3, [base], [rows], 1, group, D, 64, sharp=1.0)
    put_scales(c, 0, 0, base + rows, large)
    put_scales(c, 0, 0, base, torch.where(torch.arange(base, device="cuda") % 3 > 0, small, large)[:, None])
    got = np64(A.call(c, q, offsets, [base], None, rows))
    check_request(as_numpy(c), 0, np64(q), got, base, D ** -0.5)


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("rows,heads,D", [(1, 4, 64), (8, 8, 128), (30, 4, 128), (64, 16, 64)])
def test_drafted_rows_behind_a_cleared_context(rows, heads, D, dtype):
    """A context of a cache as it was created, and drafted rows behind it."""
    g = A.gen(1)
    table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
    c = T.KvCache.create(40, 16, 2, D, table, dtype=dtype)
    k, v = (torch.randn((2 * rows, 2, D), generator=g, device="cuda").to(BF16) for _ in range(2))
    q = torch.randn((2 * rows, heads, D), generator=g, device="cuda").to(BF16)
    at = np.arange(2 * rows)
    T.cache_write(c, k, v, i32(at // rows), i32(at % rows), base=i32([0, 200]))
    out = A.call(c, q, [0, rows, 2 * rows], [0, 200], None, rows)
    A.check(c, q, [0, rows, 2 * rows], [0, 200], None, out)


@pytest.mark.parametrize("what", ["scale", "code"])
def test_nan_in_a_drafted_row_beside_rows_of_zeros(what):
    """What a row does not see stays away from it where the sums have references of their own."""
    base, rows, group, D = 150, 6, 4, 64
    c, q, offsets, _ = A.setup(11, E4M3, [base], [rows], 1, group, D, 16, sharp=1.0)
    put_scales(c, 0, 20, 60, 0.0, True)
    words = np.array([1, 3, 0b101, 0b1001, 0b10011, 0b100101], dtype=np.uint64)
    clean = np64(A.call(c, q, offsets, [base], words, rows))
    page, slot = int(c.table[0, (base + 1) // 16]), (base + 1) % 16
    if what == "scale":
        c.v_scale[page, 0, slot] = float("nan")
    else:
        c.v.view(torch.uint8)[page, 0, slot, 3] = 0x7F
    got = np64(A.call(c, q, offsets, [base], words, rows))
    for j in range(rows):
        if j in (1, 4):  # the rows that see it
            assert np.isnan(got[j] if what == "scale" else got[j, :, 3]).all()
        else:
            np.testing.assert_array_equal(got[j], clean[j])
