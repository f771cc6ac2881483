"""GPU parity of tree_attention at the ends of its ranges.  Tolerances as in test_gpu_tree_attention.py."""
import numpy as np
import pytest
import torch

import test_gpu_tree_attention as A
from draft_sampling_lossless_markov_gb300 import capi
from draft_sampling_lossless_markov_gb300 import torch_api as T
from gpu_common import require_gpu
from kv_common import BF16, E4M3, i32

pytestmark = pytest.mark.gpu

FORMS = [(2, 2, 64), (1, 16, 128), (8, 4, 128), (4, 5, 64), (16, 4, 128), (9, 7, 64)]  # rows, heads, head size: 16, 32, 64 columns


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def set_scores(c, q, scores):
    """q and k of request 0's tokens such that every row's score of token t is scores[t], to the rounding of k (one head)."""
    D, page = c.head_dim, c.k.shape[2]
    n = scores.numel()
    q[:] = 0
    q[..., 0] = 4.0
    want = scores.cuda().float() * D ** 0.5 / 4
    t = torch.arange(n, device="cuda")
    pages, slots = c.table[0].long()[t // page], t % page
    there = pages < c.k.shape[0]
    pages, slots, want = pages[there], slots[there], want[there]
    if c.k.dtype == BF16:
        c.k[pages, 0, slots, 0] = want.to(BF16)
    else:
        scale = torch.where(want != 0, want.abs() / 448, torch.ones_like(want))
        c.k_scale[pages, 0, slots] = scale
        codes = c.k[pages, 0, slots].float()
        codes[:, 0] = want / scale
        c.k.view(torch.uint8)[pages, 0, slots] = codes.clamp(-448, 448).to(E4M3).view(torch.uint8)


def call_many(c, q, base, rows, B=608):
    """The call for so many requests like the one of c that whole items fall to a CTA; what some of them got, the workspace."""
    many = T.KvCache(c.k, c.v, c.table.expand(B, -1).contiguous(), *(() if c.k_scale is None else (c.k_scale, c.v_scale)))
    ws = T.tree_attention_workspace(B, rows, q.shape[1], 1, c.head_dim)
    out = T.tree_attention(ws, many, q.repeat(B, 1, 1), i32(np.arange(B + 1) * rows), i32([base] * B), rows)
    return [out[r * rows:(r + 1) * rows] for r in (0, 1, 2, 303, B - 1)], ws


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("rows,group,D", FORMS)
@pytest.mark.parametrize("missing", [1, 2, 3])
def test_low_scores_behind_missing_pages(missing, rows, group, D, dtype):
    """The first tiles' pages are not there, and the first scores that are seen are far below 0."""
    base, page = 900, 128
    c, q, offsets, _ = A.setup(1, dtype, [base], [rows], 1, group, D, page, fill="normal")
    q = q.clone()
    c.table[0, :missing] = 2 ** 30
    set_scores(c, q, -110 - torch.arange(base + rows) / 500)
    out, ws = call_many(c, q, base, rows)
    assert ws.read_error()[0] == capi.DSPARK_BAD_INPUT
    for o in out:
        A.check(c, q, offsets, [base], None, o)


@pytest.mark.parametrize("rows,group,D", FORMS)
@pytest.mark.parametrize("size", [2.0 ** 40, 2.0 ** 90, 2.0 ** 115, 2.0 ** -110])
@pytest.mark.parametrize("rise", [0.0, 8.0, 38.0])
def test_large_values_behind_low_scores(rise, size, rows, group, D):
    """A bf16 cache with values of one size, and scores that rise after the first tiles, so that weights pass 1."""
    base = 1100
    c, q, offsets, _ = A.setup(2, BF16, [base], [rows], 1, group, D, 64, fill="normal")
    q = q.clone()
    set_scores(c, q, torch.where(torch.arange(base + rows) < 300, 0.0, rise))
    c.v.mul_(size)
    out, ws = call_many(c, q, base, rows)
    assert ws.read_error()[0] == capi.DSPARK_OK
    for o in out:
        A.check(c, q, offsets, [base], None, o)


@pytest.mark.parametrize("rows,group,D", [(1, 16, 128), (8, 4, 128), (2, 2, 64), (16, 4, 128), (9, 7, 64)])
@pytest.mark.parametrize("n,gap", [(12000, 9), (60000, 14), (60000, 16), (250000, 16), (250000, 18)])
def test_one_token_far_above_a_long_tail(n, gap, rows, group, D):
    """e4m3: a first token `gap` above n others whose values have one sign, whole in a CTA's share.

    Of a token's weight times its scale of v (1 here), 2^-8 may be off and 2^-28 of the row's largest; all of them may be
    off to one side.  With T the tail's part of the softmax, u its value and f the first's, the result is
    f + (u - f) T; besides the rounded result the error is at most (|f| (1 - T) + |u| T) 2^-8 + n 2^-28 |u| (1 - T)."""
    page, B = 128, 304
    pages = -(-(n + rows) // page)
    k = torch.zeros((pages, 1, page, D), device="cuda")
    k[0, 0, 0, 0] = 1.0
    first = torch.tensor([0.0, 1.0, -1.0, 0.125, 16.0, 2.0 ** -6, 2.0, -4.0], device="cuda").repeat(D // 8)
    u = torch.tensor([1.0, 1.0, 1.0, -1.0, 0.5, 0.75, -2.0, 1.5], device="cuda").repeat(D // 8)
    v = u.expand(pages, 1, page, D).clone()
    v[0, 0, 0] = first
    one = torch.ones((pages, 1, page), device="cuda")
    c = T.KvCache(k.to(E4M3), v.to(E4M3), i32(np.tile(np.arange(pages), (B, 1))), one, one.clone())
    q = torch.zeros((B * rows, group, D), dtype=BF16, device="cuda")
    q[..., 0] = gap
    ws = T.tree_attention_workspace(B, rows, group, 1, D)
    out = T.tree_attention(ws, c, q, i32(np.arange(B + 1) * rows), i32([n] * B), rows, scale=1.0)
    assert ws.read_error()[0] == capi.DSPARK_OK
    tail = (n + torch.arange(rows, device="cuda", dtype=torch.float64))[:, None, None] * np.exp(-float(gap))  # and the first token: 1
    tail, first, u = tail / (1 + tail), first.double(), u.double()
    want = first + (u - first) * tail
    slack = (first.abs() * (1 - tail) + u.abs() * tail) * 2.0 ** -8 + (n + rows) * 2.0 ** -28 * u.abs() * (1 - tail) \
        + 2.0 ** -8 * want.abs() + 2.0 ** -40
    off = (out.view(B, rows, group, D).double() - want).abs()
    assert (off <= slack).all(), (off / slack).amax((0, 1, 2))[:8].tolist()
    if gap > 9:  # a tail of which nothing is lost: to 2^-7 of it and n 2^-28
        off, part = off[..., 0::8], tail.squeeze(-1)[..., None]
        assert (off <= part * 2.0 ** -7 + (n + rows) * 2.0 ** -28).all()


@pytest.mark.parametrize("rows,group,D", FORMS)
@pytest.mark.parametrize("at", [0, 130, 400, "drafted", "all"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinite_scores(sign, at, rows, group, D):
    """An infinity in k of a bf16 cache: a score of plus infinity makes a row of a head NaN, minus infinity is a weight of
    0, and a row that has no others gets 0; an element of q that is 0 there makes NaN."""
    base, page = 500, 32
    c, q, offsets, _ = A.setup(3, BF16, [base], [rows], 1, group, D, page, fill="normal", sharp=1.0)
    q = q.clone()
    q[..., 5] = 1.0
    q[:, 1::2, 5] = -1.0
    q[rows - 1, 0, 5] = 0.0
    tokens = np.arange(base + rows) if at == "all" else np.array([base if at == "drafted" else at])
    t = torch.from_numpy(tokens).cuda()
    pages, slots = c.table[0].long()[t // page], t % page
    c.k[pages, 0, slots, 5] = 0.0
    ref = A.as_numpy(c)
    c.k[pages, 0, slots, 5] = sign * float("inf")
    got = A.np64(A.call(c, q, offsets, [base], None, rows))
    k, v = (A.O.rows(ref, n, 0, range(base + rows))[:, 0] for n in ("k", "v"))
    s = D ** -0.5 * np.einsum("jgd,td->jgt", A.np64(q), k)
    direction = sign * np.sign(A.np64(q)[..., 5])
    for j in range(rows):
        seen = np.arange(base + rows) <= base + j
        hit = seen & np.isin(np.arange(base + rows), tokens)
        for g in range(group):
            if hit.any() and direction[j, g] >= 0:
                assert np.isnan(got[j, g]).all()
                continue
            use = seen & ~hit
            if not use.any():
                assert (got[j, g] == 0).all()
                continue
            e = np.exp(s[j, g, use] - s[j, g, use].max())
            want = e @ v[use] / e.sum()
            assert np.linalg.norm(got[j, g] - want) < A.NORM * np.linalg.norm(want)
