"""Sums over long peaked rows: token_logprobs keeps what small terms add to a sum that a few large ones began.

The rows begin with the largest logit in every eighth pair of their first 2048 places, so that every thread's sums begin
with it, and hold terms of 2^-24.2 of it everywhere else.  Bounds, derived before the first run: a thread adds at most
16 terms of a chunk, then the chunks (V / 4096 with 128 threads and bf16, V / 4096 with 256 and fp32, V / 8192 with 256
and bf16), then at most 16 sums of others; each addition of positive terms loses at most 2^-24 of the sum.  With
n = 32 + V / 4096 and E the mean over p, the tolerance of S is 2^-21 E(1 + |t|) + n 2^-24, of ln p the same and
2^-22 |ln p|, of the entropy 2^-21 E(1 + |t|)^2 + n 2^-24 (1 + H)."""
import numpy as np
import pytest
import torch

from draft_sampling_lossless_markov_gb300 import torch_api as T
from gpu_common import check_no_error, require_gpu
from oracle import vocab as O

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("top", [0, 3])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("offset,temp", [(0.0, 1.0), (float(2 ** 24), 1.0)])  # the second: logits too large for c x - r
@pytest.mark.parametrize("N,V", [(1, 151936), (450, 151936), (1520, 151936), (250, 1000000), (2, 2097152)])
def test_peaked_rows(N, V, offset, temp, dtype, top):
    if offset and dtype is BF16:
        pytest.skip("bf16 holds no two logits 17 apart there")
    row = torch.full((V,), offset - 17.0 if offset else -16.75, dtype=torch.float64)
    row[:2048] = row[:2048].view(-1, 8).index_fill(1, torch.tensor([0, 1]), offset).view(-1)
    z = row.to(dtype).cuda().repeat(N, 1)
    assert bool((z[0].double().cpu() == row).all())
    tok = torch.full((N,), V - 1, dtype=torch.int32, device="cuda")
    tok[::2] = 8
    ws = T.token_logprobs_workspace(N, V, top)
    got = T.token_logprobs(ws, z, tok, temp=torch.full((N,), temp, device="cuda"), top=top)
    check_no_error(ws)
    n = min(N, 2)
    ref = O.token_logprobs(row.numpy()[None].repeat(n, 0), tok[:n].cpu().numpy(), np.full(n, temp), top)
    t = (row.numpy() - offset) / temp / np.log(2)
    p = np.exp2(t)
    p /= p.sum()
    e1, e2 = (p * (1 + np.abs(t))).sum(), (p * (1 + np.abs(t)) ** 2).sum()
    walk = (32 + V / 4096) * 2.0 ** -24
    tol = 2.0 ** -21 * e1 + walk
    for k, bound in (("logprob", tol + 2.0 ** -22 * np.abs(ref["logprob"])),
                     ("top_logprob", tol + 2.0 ** -22 * np.abs(ref["top_logprob"])),
                     ("entropy", 2.0 ** -21 * e2 + walk * (1 + ref["entropy"]))):
        assert (np.abs(got[k][:n].double().cpu().numpy() - ref[k]) <= bound).all(), (k, got[k][:n], ref[k], bound)
    S = got["row_stat"][:n, 1].double().cpu().numpy()
    assert (np.abs(S / ref["row_stat"][:, 1] - 1) <= tol).all(), (S, ref["row_stat"][:, 1], tol)
    for k in ("rank", "top_id"):
        np.testing.assert_array_equal(got[k][:n].cpu().numpy(), ref[k])
    for k, v in got.items():  # equal rows, equal bits
        assert torch.equal(v[::2], v[:1].expand_as(v[::2])) and torch.equal(v[1::2], v[1:2].expand_as(v[1::2])), k
