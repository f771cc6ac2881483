"""token_logprobs and its gradient at the shapes of a full step: many rows, each walked by one CTA in many chunks, the
largest elements of a thread kept for groups of several chunks.  A sample of the rows against the fp64 oracle, with the
bounds of the row tests (their derivation holds for any length)."""
import numpy as np
import pytest
import torch

from draft_sampling_lossless_markov_gb300 import torch_api as T
from gpu_common import check_no_error, require_gpu
from test_gpu_vocab_ops import _check_grad, _check_logprobs

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _places(V):
    """Places on both sides of every boundary a CTA's walk can have (chunks of 4096 and 8192, groups of them, the ends)."""
    at = {0, 1, 6, 7, 8, V - 1, V - 2, V - 8, V - 9, V // 2}
    for e in (4096, 8192):
        last = (V - 9) // e * e
        for c in (e, 2 * e, 3 * e, 5 * e, last - e, last):
            at.update((c - 1, c, c + 5, c + e // 2))
    return np.array(sorted(p for p in at if 0 <= p < V))


def _case(N, V, dtype, shift, masked, seed):
    """Logits [N, V] whose rows begin `shift` elements past a wider row's; planted values stand above the others, in
    an order of their own in every row, some of them equal."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    wide = torch.empty((N, V + 16), dtype=dtype, device="cuda")
    z = wide[:, shift:shift + V]
    for i in range(0, N, 256):
        n = min(256, N - i)
        z[i:i + n] = (torch.randn((n, V), generator=g, device="cuda") * 1.5).to(dtype)
    at = _places(V)
    order = np.argsort(rng.random((N, at.size)), axis=1) // 2 * 2 * 0.0625 + 9.0  # pairs of equal values
    z[:, torch.from_numpy(at).cuda()] = torch.from_numpy(order).cuda().to(dtype)
    tok = np.where(rng.random(N) < 0.5, at[rng.integers(0, at.size, N)], rng.integers(0, V, N))
    tok[::11] = -1
    temp = rng.choice([0.0, 0.5, 1.0, 2.0], N).astype(np.float32)
    mask = None
    if masked:
        mask = torch.randint(-2 ** 31, 2 ** 31, (N, -(-V // 32)), generator=g, device="cuda").to(torch.int32)
        mask[3] = 0
        mask[5] = 0
        mask[5, (V - 1) >> 5] = 1 << ((V - 1) & 31) if (V - 1) & 31 < 31 else -2 ** 31
        mask[7] = -1
    rows = np.unique(np.concatenate([[0, 1, 3, 5, 7, 8, N - 1], rng.integers(0, N, 5)]))
    return z, tok, temp, mask, rows


def _forward(z, tok, temp, top, mask):
    ws = T.token_logprobs_workspace(*z.shape, top)
    out = T.token_logprobs(ws, z, torch.from_numpy(tok.astype(np.int32)).cuda(), temp=torch.from_numpy(temp).cuda(), top=top,
                           mask=mask)
    check_no_error(ws)
    return out


def _np(t, rows):
    return t[torch.from_numpy(rows).cuda()].double().cpu().numpy()


def _words(mask, rows):
    return None if mask is None else mask.cpu().numpy()[rows].view(np.uint32)


SHAPES = [(2000, 150000, BF16, 0), (2000, 150000, BF16, 3), (1600, 151936, BF16, 0), (420, 300001, BF16, 5),
          (1000, 100003, F32, 0), (1100, 50000, F32, 1), (401, 700000, F32, 2), (700, 33000, BF16, 1)]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("N,V,dtype,shift", SHAPES)
def test_rows_of_a_full_step(N, V, dtype, shift, masked):
    z, tok, temp, mask, rows = _case(N, V, dtype, shift, masked, N + V)
    at = torch.from_numpy(rows).cuda()
    for top in (0, 8, 32):
        out = _forward(z, tok, temp, top, mask)
        _check_logprobs({k: v[at] for k, v in out.items()}, _np(z, rows), tok[rows], temp[rows], top, _words(mask, rows))
        again = _forward(z, tok, temp, top, mask)
        for k in out:
            assert torch.equal(out[k].view(torch.int32), again[k].view(torch.int32)), k


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("N,V,dtype,shift", SHAPES[:1] + SHAPES[3:6])
def test_gradient_of_a_full_step(N, V, dtype, shift, masked):
    z, tok, temp, mask, rows = _case(N, V, dtype, shift, masked, 2 * N + V)
    at = torch.from_numpy(rows).cuda()
    rng = np.random.default_rng(V)
    fwd = _forward(z, tok, temp, 8, mask)
    g = [rng.standard_normal(s).astype(np.float32) for s in ((N,), (N,), (N, 8))]
    dev = [torch.from_numpy(x).cuda() for x in g]
    kw = dict(entropy=fwd["entropy"], top_id=fwd["top_id"], g_logprob=dev[0], g_entropy=dev[1], g_top=dev[2],
              temp=torch.from_numpy(temp).cuda(), mask=mask)
    ids = torch.from_numpy(tok.astype(np.int32)).cuda()
    d = T.token_logprobs_grad(None, z, ids, fwd["row_stat"], **kw)
    _check_grad(d[at], _np(z, rows), tok[rows], temp[rows], {k: v[at] for k, v in fwd.items()},
                [x[rows].astype(np.float64) for x in g], _words(mask, rows))
    if shift == 0:
        T.token_logprobs_grad(None, z, ids, fwd["row_stat"], out=z, **kw)
        assert torch.equal(z, d)
