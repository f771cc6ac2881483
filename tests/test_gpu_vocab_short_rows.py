"""token_logprobs where few of a CTA's threads hold all the candidates (short rows, masks that leave one range),
and where very many candidates tie: ids and ranks exact, log probabilities within the bounds of the row tests'
derivation (below 2^-20 of 1 + |ln p| at these lengths: |t| < 64, V < 2^14 terms)."""
import numpy as np
import pytest
import torch

from draft_sampling_lossless_markov_gb300 import torch_api as T
from gpu_common import check_no_error, require_gpu
from oracle import vocab as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _check(z, tok, top, bits=None):
    N, V = z.shape
    mask = None
    if bits is not None:
        words = np.zeros((N, -(-V // 32) * 32), dtype=np.uint8)
        words[:, :V] = bits
        packed = np.packbits(words, axis=1, bitorder="little").view(np.int32)
        mask = torch.from_numpy(packed.copy()).cuda()
    ws = T.token_logprobs_workspace(N, V, top)
    got = T.token_logprobs(ws, z, torch.from_numpy(tok.astype(np.int32)).cuda(), top=top, mask=mask)
    torch.cuda.synchronize()
    check_no_error(ws)
    y = z.double().cpu().numpy()
    if bits is not None:
        y = np.where(bits, y, -np.inf)
    ref = O.token_logprobs(y, tok, np.ones(N), top)
    np.testing.assert_array_equal(got["top_id"].cpu().numpy(), ref["top_id"])
    np.testing.assert_array_equal(got["rank"].cpu().numpy(), ref["rank"])
    for k in ("logprob", "top_logprob"):
        a, b = got[k].double().cpu().numpy(), ref[k]
        fin = np.isfinite(b)
        np.testing.assert_array_equal(a[~fin], b[~fin])
        assert (np.abs(a[fin] - b[fin]) <= 2.0 ** -18 * (1 + np.abs(b[fin]))).all()


@pytest.mark.parametrize("N", [1, 40, 700, 2100])
@pytest.mark.parametrize("V", [1, 31, 100, 260, 501, 1073, 2050])
@pytest.mark.parametrize("top", [1, 5, 32])
def test_short_rows(N, V, top):
    g = torch.Generator(device="cuda").manual_seed(V + top)
    z = torch.randn((N, V), generator=g, device="cuda")
    z = z.to(torch.bfloat16) if N % 100 else z
    _check(z, np.arange(N) % V, top)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lo,width", [(0, 300), (7, 1000), (4001, 2500), (3000, 8)])
def test_one_range_of_candidates(dtype, lo, width):
    N, V = 600, 9000
    g = torch.Generator(device="cuda").manual_seed(lo)
    z = torch.randn((N, V), generator=g, device="cuda").to(dtype)
    bits = np.zeros((N, V), dtype=bool)
    bits[:, lo:lo + width] = True
    bits[::7] = False
    _check(z, np.full(N, lo + width // 2), 20, bits)


@pytest.mark.parametrize("V", [1073, 2500, 9000])
@pytest.mark.parametrize("levels", [1, 2, 9])
def test_ties(V, levels):
    N = 450
    g = torch.Generator(device="cuda").manual_seed(levels)
    z = torch.randint(0, levels, (N, V), generator=g, device="cuda").float()
    _check(z, (np.arange(N) * 37) % V, 32)
    _check(z[:3].contiguous(), np.arange(3), 32)
