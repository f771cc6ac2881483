"""GPU parity of the vocabulary projection (quant_fp8, matmul_fp8) and of token_logprobs and its gradient
against the fp64 oracle.

Tolerances, derived before the first run:

* quant: two roundings of 2^-24 between the code and its definition, so the code lies between the e4m3
  roundings of (1 -+ 2^-22) times the exact quotient; the scale is one fp32 division (2^-24).
* matmul: products of e4m3 codes are exact in fp32; 128 additions a block, each losing at most 2^-23 of the sum
  of magnitudes (truncation allowed), then one product of scales, one product and one addition a block (2^-24
  each); a bf16 result rounds once more (half an ulp, at most 2^-8).  Integer operands whose sums stay below 2^24 must be exact.
* log probabilities: t = (logit - m) / T in base 2 carries 2^-22 |t| from three roundings, 2^t another 2^-22, and
  sums of up to V / 128 terms in a row a random walk of 2^-24 steps (6 sigma).  With E the mean over p:
  tol_S = 2^-21 E(1 + |t|) + 6 sqrt(V / 128) 2^-24, logprob tol_S + 2^-22 |logprob|, entropy
  2^-21 E(1 + |t|)^2 + 6 sqrt(V / 128) 2^-24 (1 + H).
* gradient: p carries tol_S + 2^-21 (1 + |t|) relative; each term of the formula 2^-21 more; a bf16 result
  2^-8.
"""
import numpy as np
import pytest
import torch

from oracle import vocab as O
from draft_sampling_lossless_markov_gb300 import capi
from draft_sampling_lossless_markov_gb300 import torch_api as T
from gpu_common import check_no_error, require_gpu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def np64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def codes_np(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int64).astype(np.uint32).view(np.int32)).cuda()


# --------------------------------------------------------------------------- quant
def _check_quant(x, block_rows, codes, scale):
    exact, want = O.quant(np64(x), block_rows)
    got = O.e4m3_decode(codes_np(codes))
    nan = np.isnan(exact)
    np.testing.assert_array_equal(np.isnan(got), nan)
    lo, hi = O.e4m3_round(exact[~nan] * (1 - 2.0 ** -22)), O.e4m3_round(exact[~nan] * (1 + 2.0 ** -22))
    assert ((np.minimum(lo, hi) <= got[~nan]) & (got[~nan] <= np.maximum(lo, hi))).all()
    np.testing.assert_allclose(np64(scale), want, rtol=2.0 ** -23)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 128), (3, 127), (129, 129), (5, 1000), (300, 520), (128, 4096)])
def test_quant(M, K, dt, block_rows):
    g = torch.Generator().manual_seed(M * 10007 + K)
    x = (torch.randn((M, K), generator=g) * torch.exp(2 * torch.randn((M, 1), generator=g))).to(dt).cuda()
    codes, scale = T.quant_fp8(x, block_rows)
    _check_quant(x, block_rows, codes, scale)


def test_quant_zero_tiny_and_non_finite_blocks():
    x = torch.randn(6, 300).cuda()
    x[0] = 0
    x[1, :128] = 1e-38
    x[2, 5], x[2, 130], x[3, 299] = float("nan"), float("inf"), float("-inf")
    x[4, 7] = 3.0e38
    x[5, :128] = -0.0
    for rows in (1, 128):
        codes, scale = T.quant_fp8(x, rows)
        _check_quant(x, rows, codes, scale)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quant_strided_and_misaligned(dt, block_rows):
    base = torch.randn(200, 517, device="cuda").to(dt)
    store = torch.zeros((200, 600), dtype=torch.uint8, device="cuda")
    for c0, c1 in ((0, 256), (3, 400), (8, 517)):
        x = base[:, c0:c1]
        store.fill_(0x55)
        codes = store[:, 1:1 + c1 - c0].view(torch.float8_e4m3fn)
        scale = torch.empty((200 if block_rows == 1 else 2, -(-(c1 - c0) // 128)), device="cuda")
        T.quant_fp8(x, block_rows, out=(codes, scale))
        _check_quant(x, block_rows, codes, scale)
        assert bool((store[:, :1] == 0x55).all()) and bool((store[:, 1 + c1 - c0:] == 0x55).all())


def test_quant_no_rows():
    codes, scale = T.quant_fp8(torch.empty((0, 300), device="cuda"))
    assert codes.shape == (0, 300) and scale.shape == (0, 3)


# --------------------------------------------------------------------------- matmul
def _codes_of(x):
    """Dense e4m3 values to codes with the row stride matmul needs."""
    q = T.fp8_codes(*x.shape)
    q.copy_(x.to(torch.float8_e4m3fn))
    return q


def _random_operands(M, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = _codes_of(torch.randn((M, K), generator=g, device="cuda") * 60)
    w = _codes_of(torch.randn((N, K), generator=g, device="cuda") * 60)
    kb = -(-K // 128)
    sa = torch.exp(torch.randn((M, kb), generator=g, device="cuda") * 2) * 0.01
    sw = torch.exp(torch.randn((-(-N // 128), kb), generator=g, device="cuda") * 2) * 0.01
    return a, sa, w, sw


def _check_matmul(out, a, sa, w, sw, rows=None):
    y, mag = O.matmul(codes_np(a), np64(sa), codes_np(w), np64(sw))
    kb = sa.shape[1]
    tol = (128 * 2.0 ** -23 + (kb + 3) * 2.0 ** -24) * mag
    if out.dtype == BF16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(y) + 1e-38
    rows = slice(0, rows)
    assert (np.abs(np64(out) - y)[rows] <= tol[rows]).all()


SHAPES = [(1, 128, 128), (1, 1, 1), (2, 127, 129), (1, 1000, 2560), (7, 300, 520), (16, 2560, 1000), (33, 129, 64),
          (64, 513, 2050), (65, 128, 384), (127, 640, 250), (128, 256, 512), (129, 257, 4096), (200, 1111, 136),
          (257, 384, 1024), (300, 1000, 2050), (513, 513, 513), (1000, 260, 200)]


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul_random_scales(M, N, K, out_dtype):
    a, sa, w, sw = _random_operands(M, N, K, M * 7 + N * 3 + K)
    ws = T.matmul_fp8_workspace(M, N, K)
    out = T.matmul_fp8(ws, a, sa, w, sw, out_dtype=out_dtype)
    check_no_error(ws)
    _check_matmul(out, a, sa, w, sw)
    again = T.matmul_fp8(ws, a, sa, w, sw, out_dtype=out_dtype)
    assert torch.equal(out, again)


@pytest.mark.parametrize("M,N,K", [(1, 640, 1000), (8, 130, 4096), (40, 384, 300), (100, 129, 2050), (300, 700, 1030),
                                   (513, 1025, 640), (2048, 300, 256)])
def test_matmul_of_whole_numbers_is_exact(M, N, K):
    # codes in -8..8, scales powers of two from 1 to 4: every sum is a whole number below 2^24
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    kb, nb = -(-K // 128), -(-N // 128)
    a = _codes_of(torch.randint(-8, 9, (M, K), generator=g, device="cuda").float())
    w = _codes_of(torch.randint(-8, 9, (N, K), generator=g, device="cuda").float())
    sa = torch.randint(0, 2, (M, kb), generator=g, device="cuda").float().exp2()
    sw = torch.randint(0, 2, (nb, kb), generator=g, device="cuda").float().exp2()
    ws = T.matmul_fp8_workspace(M, N, K)
    out = T.matmul_fp8(ws, a, sa, w, sw, out_dtype=F32)
    check_no_error(ws)
    y, _ = O.matmul(codes_np(a), np64(sa), codes_np(w), np64(sw))
    np.testing.assert_array_equal(np64(out), y)


@pytest.mark.parametrize("M,N,K", [(5, 200, 300), (150, 260, 300)])
def test_matmul_strided_operands_and_output(M, N, K):
    big_a = _codes_of(torch.randn((M, 512), device="cuda") * 50)
    big_w = _codes_of(torch.randn((N, 640), device="cuda") * 50)
    a, w = big_a[:, 32:32 + K], big_w[:, 48:48 + K]
    sa = torch.rand((M, 3), device="cuda") + 0.5
    sw = torch.rand((-(-N // 128), 3), device="cuda") + 0.5
    ws = T.matmul_fp8_workspace(M, N, K)
    for dt in (BF16, F32):
        for c0, ld in ((0, N), (3, N + 9), (8, N + 16)):
            store = torch.full((M, ld + c0), -7.0, dtype=dt, device="cuda")
            out = store[:, c0:c0 + N]
            T.matmul_fp8(ws, a, sa, w, sw, out=out)
            check_no_error(ws)
            _check_matmul(out, a, sa, w, sw)
            assert bool((store[:, :c0] == -7).all()) and bool((store[:, c0 + N:] == -7).all())


@pytest.mark.parametrize("M,count", [(10, 0), (10, 7), (300, 129), (300, 300), (300, 1000), (700, 1), (40, -3)])
def test_matmul_row_count_on_the_device(M, count):
    N, K = 500, 700
    a, sa, w, sw = _random_operands(M, N, K, M + count)
    out = torch.full((M, N), -7.0, device="cuda")
    ws = T.matmul_fp8_workspace(M, N, K)
    T.matmul_fp8(ws, a, sa, w, sw, out=out, n_rows=torch.tensor([count], dtype=torch.int32, device="cuda"))
    check_no_error(ws)
    n = max(0, min(M, count))
    if n:
        _check_matmul(out, a, sa, w, sw, n)
    assert bool((out[n:] == -7).all())


def test_matmul_nan_codes_stay_in_their_row_and_column():
    M, N, K = 20, 300, 300
    a, sa, w, sw = _random_operands(M, N, K, 5)
    a.view(torch.uint8)[3, 7] = 0x7F
    w.view(torch.uint8)[290, 299] = 0xFF
    ws = T.matmul_fp8_workspace(M, N, K)
    out = np64(T.matmul_fp8(ws, a, sa, w, sw, out_dtype=F32))
    want = np.zeros((M, N), bool)
    want[3], want[:, 290] = True, True
    np.testing.assert_array_equal(np.isnan(out), want)


def test_matmul_empty_and_other_stream_and_graph():
    ws = T.matmul_fp8_workspace(4, 4, 16)
    e = T.fp8_codes(0, 16)
    w = _codes_of(torch.ones(4, 16, device="cuda"))
    assert T.matmul_fp8(ws, e, torch.empty((0, 1), device="cuda"), w, torch.ones((1, 1), device="cuda")).shape == (0, 4)
    M, N, K = 9, 400, 900
    a, sa, w, sw = _random_operands(M, N, K, 11)
    ws = T.matmul_fp8_workspace(M, N, K)
    want = T.matmul_fp8(ws, a, sa, w, sw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    T.matmul_fp8(ws, a, sa, w, sw, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        T.matmul_fp8(ws, a, sa, w, sw, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# --------------------------------------------------------------------------- token log probabilities
def _row_bounds(z, temp, mask):
    """Per row: E(1 + |t|), E(1 + |t|)^2 under p, and the walk of the sums."""
    ok = O.candidates(z, mask)
    Tt = O.temperature(temp)[:, None]
    e1, e2 = np.ones(len(z)), np.ones(len(z))
    for i in range(len(z)):
        x = z[i, ok[i]]
        if x.size and np.isfinite(x).all():
            t = (x - x.max()) / Tt[i] / np.log(2)
            p = np.exp2(t)
            p /= p.sum()
            e1[i], e2[i] = (p * (1 + np.abs(t))).sum(), (p * (1 + np.abs(t)) ** 2).sum()
    return e1, e2, 6 * np.sqrt(z.shape[1] / 128) * 2.0 ** -24


def _close(got, want, tol, what):
    got, want, tol = np.asarray(got), np.asarray(want), np.broadcast_to(tol, np.shape(want))
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want), err_msg=what)
    fin = np.isfinite(want)
    np.testing.assert_array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)], err_msg=what)
    bad = np.abs(got[fin] - want[fin]) > tol[fin]
    assert not bad.any(), (what, np.abs(got[fin] - want[fin])[bad].max(), bad.sum())


def _check_logprobs(out, z, tok, temp, top, mask=None, rows=slice(None)):
    with np.errstate(over="ignore"):
        ref = O.token_logprobs(z, tok, temp, top, mask)
        e1, e2, walk = _row_bounds(z, temp, mask)
    got = {k: (v.cpu().numpy() if v.dtype == torch.int32 else np64(v))[rows] for k, v in out.items()}
    with np.errstate(over="ignore"):  # a log probability past fp32's range is -inf
        ref = {k: np.where(np.abs(v) > 3.4e38, np.float32(v), v)[rows] for k, v in ref.items()}
    e1, e2 = e1[rows], e2[rows]
    tol_s = 2.0 ** -21 * e1 + walk
    np.testing.assert_array_equal(got["rank"], ref["rank"])
    np.testing.assert_array_equal(got["top_id"], ref["top_id"])
    fin = lambda v: np.where(np.isfinite(v), np.abs(v), 0)  # noqa: E731
    _close(got["logprob"], ref["logprob"], tol_s + 2.0 ** -22 * fin(ref["logprob"]), "logprob")
    _close(got["top_logprob"], ref["top_logprob"], tol_s[:, None] + 2.0 ** -22 * fin(ref["top_logprob"]), "top_logprob")
    _close(got["entropy"], ref["entropy"], 2.0 ** -21 * e2 + walk * (1 + fin(ref["entropy"])), "entropy")
    good = ~np.isnan(ref["row_stat"][:, 1])
    np.testing.assert_array_equal(got["row_stat"][good, 0], ref["row_stat"][good, 0])
    _close(got["row_stat"][:, 1], ref["row_stat"][:, 1], tol_s * fin(ref["row_stat"][:, 1]), "S")
    return ref


def _logits(N, V, dt, seed, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((N, V), generator=g) * scale - 1.1 * torch.log(torch.arange(V) + 1.0)
    return z.to(dt).cuda()


def _tokens(N, V, seed):
    rng = np.random.default_rng(seed)
    tok = rng.integers(0, V, N)
    tok[rng.random(N) < 0.2] = -1
    temp = rng.choice([0.0, 0.3, 0.7, 1.0, 2.0, -1.0, np.nan, np.inf], N).astype(np.float32)
    return tok, temp


def _run(z, tok, temp, top, mask=None, **kw):
    ws = T.token_logprobs_workspace(z.shape[0], z.shape[1], top)
    out = T.token_logprobs(ws, z, i32(tok), temp=None if temp is None else torch.from_numpy(temp).cuda(), top=top,
                           mask=None if mask is None else i32(mask), **kw)
    check_no_error(ws)
    return out


LP = [(1, 1, 0), (1, 1, 5), (3, 2, 1), (2, 31, 32), (5, 33, 20), (4, 255, 3), (3, 257, 32), (7, 1000, 8), (2, 4099, 5),
      (1, 50001, 20), (9, 30011, 0), (300, 2048, 4), (1, 151936, 32), (3, 129280, 8), (40, 151936, 1)]


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("N,V,top", LP)
def test_logprobs(N, V, top, dt):
    z = _logits(N, V, dt, N + V)
    tok, temp = _tokens(N, V, N * 3 + V)
    out = _run(z, tok, temp, top)
    _check_logprobs(out, np64(z), tok, temp, top)
    again = _run(z, tok, temp, top)
    for k in out:
        assert torch.equal(out[k], again[k]), k


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("N,V,top", [(6, 40, 5), (9, 1000, 20), (5, 30011, 8), (3, 151936, 32), (33, 4096, 0)])
def test_logprobs_masked(N, V, top, dt):
    rng = np.random.default_rng(V)
    z = _logits(N, V, dt, V)
    W = -(-V // 32)
    mask = rng.integers(0, 2 ** 32, (N, W + 2), dtype=np.uint64) & rng.integers(0, 2 ** 32, (N, W + 2), dtype=np.uint64)
    mask[0] = 0                      # nothing left
    mask[1] = 0
    mask[1, (V - 1) >> 5] = 1 << ((V - 1) & 31)  # the last place alone
    mask[2] = 0xFFFFFFFF
    tok, temp = _tokens(N, V, V)
    tok[0], tok[1] = 0, V - 1
    # masked places may hold anything
    ok = O.candidates(np.zeros((N, V)), mask)
    junk = torch.from_numpy(rng.choice([np.nan, np.inf, -np.inf, 3e38], (N, V)).astype(np.float32)).cuda().to(dt)
    z = torch.where(torch.from_numpy(ok).cuda(), z, junk)
    out = _run(z, tok, temp, top, mask)
    _check_logprobs(out, np64(z), tok, temp, top, mask)


@pytest.mark.parametrize("V", [100, 3000, 40000])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_logprobs_special_values(V, dt):
    lowest = float(torch.finfo(dt).min)
    z = _logits(12, V, dt, 7)
    z[0] = float("-inf")
    z[1] = lowest                                   # a uniform row of the lowest value
    z[2, 1:] = lowest
    z[3, ::2] = float("-inf")
    z[4, V // 2] = float("nan")
    z[5, V - 1] = float("inf")
    z[6] = 0.0
    z[6, 1::2] = -0.0                               # one tie over the whole row
    z[7] = torch.arange(V, device="cuda").to(dt)   # ascending: every place is a new best
    z[8] = -torch.arange(V, device="cuda").to(dt)
    z[9, : V - 1] = float("-inf")
    z[10] = z[10].abs() * 1e4
    z[11] = float("-inf")
    z[11, 3], z[11, 7] = lowest, lowest
    tok = np.array([3, 5, 0, 1, 2, 1, V - 1, 0, V - 1, V - 1, 4, 7])
    for temp in (np.ones(12, np.float32), np.full(12, 0.25, np.float32), np.full(12, 1e-30, np.float32),
                 np.full(12, 1e30, np.float32)):
        out = _run(z, tok, temp, 20)
        _check_logprobs(out, np64(z), tok, temp, 20)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_logprobs_strided_misaligned_and_partial_outputs(dt):
    N, V = 6, 5003
    base = _logits(N, V + 13, dt, 9)
    tok, temp = _tokens(N, V, 4)
    for c0 in (0, 1, 5, 8):
        z = base[:, c0:c0 + V]
        _check_logprobs(_run(z, tok, temp, 7), np64(z), tok, temp, 7)
    z = base[:, :V]
    full = _run(z, tok, temp, 0)
    ent = torch.zeros(N, device="cuda")
    _run(z, tok, temp, 0, out=dict(entropy=ent))
    assert torch.equal(ent, full["entropy"])
    one = _run(z, tok, None, 0)
    _check_logprobs(one, np64(z), tok, np.ones(N, np.float32), 0)


def test_logprobs_markers_row_count_and_bad_input():
    B, G1, V, N = 5, 4, 700, 17
    rng = np.random.default_rng(0)
    req = np.array([0, 0, 0, 1, 2, 2, 2, 2, 3, 3, 4, -1, -1, 9, 0, 1, 2])
    pos = np.array([0, 1, 2, 0, 0, 1, 2, 3, 0, 1, 0, -1, -1, 0, 4, -2, 0])
    table = rng.integers(0, V, (B, G1))
    table[0, 2], table[2, 3] = -1, V
    temp = np.array([0.0, 0.5, 1.0, 2.0, 0.7], np.float32)
    ok = (req >= 0) & (req < B) & (pos >= 0) & (pos < G1)
    tok = np.where(ok, table[np.where(ok, req, 0), np.where(ok, pos, 0)], -1)
    tok[tok >= V] = -1
    row_t = np.where(ok, temp[np.where(ok, req, 0)], 1.0).astype(np.float32)
    z = _logits(N, V, BF16, 3)
    ws = T.token_logprobs_workspace(N, V, 3)
    for count in (None, 0, 1, 16, 99):
        out = dict(logprob=torch.full((N,), -7.0, device="cuda"), entropy=torch.full((N,), -7.0, device="cuda"),
                   rank=torch.full((N,), -7, dtype=torch.int32, device="cuda"),
                   row_stat=torch.full((N, 2), -7.0, device="cuda"),
                   top_id=torch.full((N, 3), -7, dtype=torch.int32, device="cuda"),
                   top_logprob=torch.full((N, 3), -7.0, device="cuda"))
        T.token_logprobs(ws, z, i32(table), temp=torch.from_numpy(temp).cuda(), top=3, mark_req=i32(req),
                         mark_pos=i32(pos), out=out,
                         n_rows=None if count is None else torch.tensor([count], dtype=torch.int32, device="cuda"))
        n = N if count is None else min(N, count)
        code, detail = ws.read_error()
        bad = [i for i in range(n) if i in (7, 13, 14, 15)]  # a token of V, requests and places out of range
        assert (code in (0, capi.DSPARK_BAD_INPUT)) and (code != 0) == bool(bad) and (not bad or detail in bad)
        _check_logprobs(out, np64(z), tok, row_t, 3, rows=slice(0, n))
        for t in out.values():
            assert bool((t[n:] == -7).all())


def test_logprobs_no_rows():
    ws = T.token_logprobs_workspace(0, 10, 2)
    out = T.token_logprobs(ws, torch.empty((0, 10), device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), top=2)
    assert out["top_id"].shape == (0, 2)


# --------------------------------------------------------------------------- gradient
def _grad_case(z, tok, temp, top, mask, seed, use=("l", "e", "t")):
    N = z.shape[0]
    rng = np.random.default_rng(seed)
    fwd = _run(z, tok, temp, top, mask)
    g = [rng.standard_normal(s).astype(np.float32) for s in ((N,), (N,), (N, top))]
    dev = [torch.from_numpy(x).cuda() for x in g]
    kw = dict(g_logprob=dev[0] if "l" in use else None, g_entropy=dev[1] if "e" in use else None,
              g_top=dev[2] if "t" in use and top else None, temp=torch.from_numpy(temp).cuda(),
              mask=None if mask is None else i32(mask), entropy=fwd["entropy"], top_id=fwd["top_id"])
    g = [x if u in use else np.zeros_like(x) for x, u in zip(g, ("l", "e", "t"))]
    return fwd, [x.astype(np.float64) for x in g], kw


def _check_grad(d, z, tok, temp, fwd, g, mask, rows=slice(None)):
    tid = fwd["top_id"].cpu().numpy()
    want = O.token_logprobs_grad(z, tok, temp, tid, *g, mask)
    ok, Tt = O.candidates(z, mask), O.temperature(temp)[:, None]
    e1, e2, walk = _row_bounds(z, temp, mask)
    zm = np.where(ok & np.isfinite(z), z, -np.inf)
    m = zm.max(1, keepdims=True)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        t = np.where(np.isneginf(zm), 0, np.minimum(0, (zm - np.where(np.isneginf(m), 0, m)) / Tt / np.log(2)))
        p = np.where(np.isneginf(zm), 0, np.exp2(t))
        p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
        logp = np.where(p > 0, np.log(np.maximum(p, 1e-300)), 0)
    H = -(p * logp).sum(1, keepdims=True)
    tol_s = (2.0 ** -21 * e1 + walk)[:, None]
    tol_h = (2.0 ** -21 * e2 + walk * (1 + H[:, 0]))[:, None]
    Gabs = np.abs(g[0])[:, None] + np.abs(g[2]).sum(1)[:, None]
    He = np.abs(g[1])[:, None]
    size = p * (Gabs + He * (np.abs(logp) + H))
    picked = np.zeros_like(z)
    for at, w in [(tok, g[0])] + [(tid[:, k], g[2][:, k]) for k in range(tid.shape[1])]:
        r = np.flatnonzero(at >= 0)
        picked[r, at[r]] += np.abs(w[r])
    tol = (size * (tol_s + 2.0 ** -21 * (1 + np.abs(t))) + He * p * (tol_h + tol_s + 2.0 ** -21 * (1 + np.abs(t)))
           + 2.0 ** -21 * picked * (2 + tid.shape[1])) / Tt + 1e-37
    got = np64(d)
    if d.dtype == BF16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    np.testing.assert_array_equal(got[rows][~ok[rows]], 0)
    assert (np.abs(got - want)[rows] <= tol[rows]).all(), np.max((np.abs(got - want) / tol)[rows])


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("N,V,top,masked", [(1, 1, 1, False), (3, 2, 2, False), (4, 33, 5, True), (5, 1000, 0, False),
                                            (6, 4099, 20, True), (2, 30011, 32, False), (1, 151936, 8, False),
                                            (7, 20000, 3, True), (300, 520, 1, False)])
def test_grad(N, V, top, masked, dt):
    rng = np.random.default_rng(V + N)
    z = _logits(N, V, dt, N * V)
    tok, temp = _tokens(N, V, V + 1)
    mask = None
    if masked:
        mask = rng.integers(0, 2 ** 32, (N, -(-V // 32)), dtype=np.uint64)
        mask[0] = 0
        junk = torch.full_like(z, float("nan"))
        z = torch.where(torch.from_numpy(O.candidates(np.zeros((N, V)), mask)).cuda(), z, junk)
    for use in (("l", "e", "t"), ("l",), ("e",), ("t",)):
        fwd, g, kw = _grad_case(z, tok, temp, top, mask, N + V, use)
        d = T.token_logprobs_grad(None, z, i32(tok), fwd["row_stat"], **kw)
        _check_grad(d, np64(z), tok, temp, fwd, g, mask)
    same = z.clone()
    T.token_logprobs_grad(None, same, i32(tok), fwd["row_stat"], out=same, **kw)
    assert torch.equal(same, d)


def test_grad_against_differences():
    # central differences of the fp64 loss: step 1e-5, so their own error is below 1e-8
    N, V, top = 5, 40, 4
    z = _logits(N, V, F32, 2, 1.5)
    z[1, 5] = float("-inf")
    mask = np.random.default_rng(1).integers(0, 2 ** 32, (N, 2), dtype=np.uint64) | 2
    mask[3] = 0
    tok, temp = np.array([1, 5, -1, 2, 1]), np.array([1.0, 0.5, 0.0, 1.0, 1.7], np.float32)
    fwd, g, kw = _grad_case(z, tok, temp, top, mask, 8)
    d = np64(T.token_logprobs_grad(None, z, i32(tok), fwd["row_stat"], **kw))
    x, tid, h = np64(z), fwd["top_id"].cpu().numpy(), 1e-5
    for v in range(V):
        e = np.zeros(V)
        e[v] = h
        num = (O.loss(x + e, tok, temp, tid, *g, mask) - O.loss(x - e, tok, temp, tid, *g, mask)) / (2 * h)
        np.testing.assert_allclose(d[:, v], num, atol=2e-5)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_grad_special_rows(dt):
    V = 3000
    lowest = float(torch.finfo(dt).min)
    z = _logits(7, V, dt, 5)
    z[0] = float("-inf")
    z[1] = lowest
    z[2, 1:] = lowest
    z[3, ::2] = float("-inf")
    z[4, 7] = float("nan")
    z[5] = 0.0
    z[6, :V - 1] = float("-inf")
    tok = np.array([1, 2, 0, 2, 3, 4, V - 1])
    temp = np.ones(7, np.float32)
    fwd, g, kw = _grad_case(z, tok, temp, 5, None, 3)
    d = T.token_logprobs_grad(None, z, i32(tok), fwd["row_stat"], **kw)
    assert bool(torch.isnan(d[4]).all())
    keep = [0, 1, 2, 3, 5, 6]
    cut = {k: v[keep] for k, v in fwd.items()}
    _check_grad(d[keep], np64(z[keep]), tok[keep], temp[keep], cut, [x[keep] for x in g], None)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_grad_strided_misaligned_and_row_count(dt):
    N, V = 6, 5003
    base = _logits(N, V + 13, dt, 19)
    tok, temp = _tokens(N, V, 4)
    for c0, count in ((0, None), (1, 4), (5, 0), (8, 6)):
        z = base[:, c0:c0 + V]
        fwd, g, kw = _grad_case(z, tok, temp, 3, None, c0)
        store = torch.full((N, V + 9), -7.0, dtype=dt, device="cuda")
        out = store[:, c0 // 2:c0 // 2 + V]
        n = N if count is None else count
        T.token_logprobs_grad(None, z, i32(tok), fwd["row_stat"], out=out, n_rows=None if count is None else
                              torch.tensor([count], dtype=torch.int32, device="cuda"), **kw)
        _check_grad(out, np64(z), tok, temp, fwd, g, None, slice(0, n))
        assert bool((store[:, :c0 // 2] == -7).all()) and bool((store[:, c0 // 2 + V:] == -7).all())
        assert bool((store[n:] == -7).all())


# --------------------------------------------------------------------------- cases of single paths
def test_quant_of_fp32_rounds_the_exact_quotient():
    # products that fp32 puts on the wrong side of the middle between two codes: x one
    # float from middle * amax / 448, both sides of every middle, blocks of two amax
    mids = (O.e4m3_values()[:126] + O.e4m3_values()[1:127]) / 2
    for amax in (3.0, 0.1, 7.7e-20, 5.3e30):
        base = (mids * (amax / 448)).astype(np.float32)
        rows = [base, np.nextafter(base, np.float32(0)), np.nextafter(base, np.float32(np.inf)), -base]
        x = np.concatenate([np.stack(rows), np.full((4, 2), amax, np.float32)], 1)
        assert x.shape[1] == 128
        t = torch.from_numpy(x).cuda()
        for block_rows in (1, 128):
            codes, _ = T.quant_fp8(t, block_rows)
            a = np.abs(x.astype(np.float64)).max()
            want = O.e4m3_round(x.astype(np.float64) * 448.0 / a)
            frac = x.astype(np.float64) * 448.0 / a
            tie = np.isin(np.abs(frac), mids)  # fp64 itself cannot tell: either neighbour
            got = O.e4m3_decode(codes_np(codes))
            np.testing.assert_array_equal(got[~tie], want[~tie])


def test_quant_many_rows_and_non_finite_in_some():
    # enough blocks for the wide form of the row kernel; non-finite elements in a few of them
    x = torch.randn(20000, 1700, device="cuda")
    at = torch.randint(0, x.numel(), (500,), device="cuda")
    x.view(-1)[at] = float("nan")
    x.view(-1)[at[:200]] = float("inf")
    for dt in (BF16, F32):
        y = x.to(dt)
        codes, scale = T.quant_fp8(y, 1)
        rows = torch.unique(at // 1700)[:60]
        _check_quant(y[rows], 1, codes[rows], scale[rows])


@pytest.mark.parametrize("dt", [BF16, F32])
def test_logprobs_more_ties_than_the_candidate_buffer(dt):
    # rows where thousands of places tie with the K-th: the lowest ids win
    V = 30000
    z = torch.zeros(4, V, device="cuda", dtype=dt)
    z[1, ::2] = 1.0
    z[2, 5000:] = 2.0
    z[2, 29000] = 3.0
    z[3] = torch.arange(V, device="cuda").to(dt) // 4096
    tok, temp = np.array([17, 29998, 29000, 0]), np.ones(4, np.float32)
    for top in (1, 20, 32):
        _check_logprobs(_run(z, tok, temp, top), np64(z), tok, temp, top)


@pytest.mark.parametrize("M,N,K", [(5, 900, 7168), (200, 640, 4096), (64, 384, 8192), (33, 2560, 2560)])
def test_matmul_split_over_k(M, N, K):
    a, sa, w, sw = _random_operands(M, N, K, M)
    ws = T.matmul_fp8_workspace(M, N, K)
    for dt in (BF16, F32):
        out = T.matmul_fp8(ws, a, sa, w, sw, out_dtype=dt)
        check_no_error(ws)
        _check_matmul(out, a, sa, w, sw)
