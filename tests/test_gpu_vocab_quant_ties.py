"""quant_fp8 gives every element the code of its exact quotient x 448 / amax, ties to the even code.

x and amax have 8 significant bits here, so x 448 and (middle between two codes) amax are exact in fp64 and their
comparison is the rounding's definition: no tolerance."""
import numpy as np
import pytest
import torch

from draft_sampling_lossless_markov_gb300 import torch_api as T
from gpu_common import require_gpu
from oracle import vocab as O

pytestmark = pytest.mark.gpu

POS = O.e4m3_values()[:127]
MIDDLES = (POS[:-1] + POS[1:]) / 2


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _codes(x, amax):
    """[rows, n] whole codes (sign bit included) of x with one amax a row."""
    want = np.empty(x.shape, np.uint8)
    for i, a in enumerate(amax):
        y, t = np.abs(x[i]) * 448.0, MIDDLES * a
        lo = np.searchsorted(t, y, side="left")
        tie = (lo < 126) & (t[np.minimum(lo, 125)] == y)
        want[i] = lo + (tie & (lo % 2 == 1)) + 128 * np.signbit(x[i])
    return want


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("exponent", [0, -60, -100, 90, 120])
def test_codes_of_every_pair_of_significands(dtype, exponent):
    # rows: every significand of amax; columns: every significand of x at 19 sizes below it, 127 a block beside amax
    amax = np.arange(128, 256) * 2.0 ** (exponent - 7)
    cols = (np.arange(128, 256)[:, None] * 2.0 ** (exponent - 8 - np.arange(19))[None]).ravel()
    cols[1::2] *= -1
    blocks = -(-cols.size // 127)
    cols = np.concatenate([cols, np.zeros(blocks * 127 - cols.size)]).reshape(blocks, 127)
    x = np.concatenate([np.broadcast_to(cols, (128, blocks, 127)),
                        np.broadcast_to(amax[:, None, None], (128, blocks, 1))], 2).reshape(128, blocks * 128)
    want = _codes(x, amax)
    t = torch.from_numpy(x).to(dtype).cuda()
    assert bool((t.double().cpu().numpy() == x).all())
    codes, scale = T.quant_fp8(t, 1)
    np.testing.assert_array_equal(codes.contiguous().view(torch.uint8).cpu().numpy(), want)
    np.testing.assert_array_equal(scale.cpu().numpy()[:, 0], (amax.astype(np.float32) / np.float32(448)))
    for i in (0, 33, 127):  # as one 128 x 128 block: 128 rows with one amax
        codes, _ = T.quant_fp8(t[i:i + 1].repeat(128, 1), 128)
        np.testing.assert_array_equal(codes.contiguous().view(torch.uint8).cpu().numpy(),
                                      np.broadcast_to(want[i], (128, want.shape[1])))
