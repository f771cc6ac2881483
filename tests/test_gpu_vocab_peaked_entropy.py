"""The entropy of rows with one peak, wherever it stands and however far it is above what came before it.

Bound, derived before the first run: ln S carries 2^-21 E(1 + |t|) (the exponential twice, its argument once), A / S the
same for each term's |t|, so 2^-21 E(1 + |t|)^2 together; a term above the reference of its thread's sums is one of at
most 2^4 S, rounded twice (2^-24 each) before the move to the largest element takes most of it away: 8 ln 2 2^-24 < 2^-21;
the sums' walk as in the row tests; the two numbers subtracted, 2^-23 (1 + H)."""
import numpy as np
import pytest
import torch

from draft_sampling_lossless_markov_gb300 import torch_api as T
from gpu_common import check_no_error, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("temp", [1.0, 0.5])
@pytest.mark.parametrize("N,V", [(640, 12), (640, 700), (640, 3001), (640, 151936), (1600, 60000), (3, 151936)])
def test_one_peak(N, V, temp, dtype):
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn((N, V), generator=g, device="cuda") * 0.3
    i = torch.arange(N, device="cuda")
    at = (i * 7919) % V                       # everywhere, the last place too
    at[::5] = V - 1
    z[i, at] = (6.0 + 16.0 * (i % 64) / 64 + torch.rand((N,), generator=g, device="cuda")) * temp * (1 + np.log(V) / 16)
    z = z.to(dtype)
    ws = T.token_logprobs_workspace(N, V, 0)
    tok = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    got = T.token_logprobs(ws, z, tok, temp=torch.full((N,), temp, device="cuda"))
    check_no_error(ws)
    for lo in range(0, N, 128):
        x = z[lo:lo + 128].double()
        y = (x - x.amax(1, keepdim=True)) / temp
        S = y.exp().sum(1, keepdim=True)
        p = y.exp() / S
        H = S.log()[:, 0] - (p * y).sum(1)
        t = y.abs() / np.log(2)
        e2 = (p * (1 + t) ** 2).sum(1)
        bound = 2.0 ** -21 * (e2 + 1) + 6 * (V / 128) ** 0.5 * 2.0 ** -24 * (1 + H) + 2.0 ** -23 * (1 + H)
        err = (got["entropy"][lo:lo + 128].double() - H).abs()
        assert bool((err <= bound).all()), (float((err / bound).max()), float(err.max()))
