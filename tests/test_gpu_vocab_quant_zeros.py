"""quant_fp8 keeps the sign of zeros, and of what rounds to zero, whatever the block's largest magnitude."""
import numpy as np
import pytest
import torch

from draft_sampling_lossless_markov_gb300 import torch_api as T
from gpu_common import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tiny", [0.0, 2.0 ** -120, 2.0 ** -133])
def test_signs(dtype, tiny):
    require_gpu()
    x = torch.full((128, 128), tiny, device="cuda")
    x[:, 1::2] = -x[:, 1::2]
    x[:, 0] = torch.arange(128, 256, device="cuda") * 0.37  # a largest magnitude a row
    x = x.to(dtype)
    want = np.where(np.arange(128) % 2 == 1, 128, 0)
    codes, _ = T.quant_fp8(x, 1)
    got = codes.contiguous().view(torch.uint8).cpu().numpy()
    np.testing.assert_array_equal(got[:, 1:], np.broadcast_to(want[1:], (128, 127)))
    for i in (0, 7, 70, 127):
        codes, _ = T.quant_fp8(x[i:i + 1].repeat(128, 1), 128)
        got = codes.contiguous().view(torch.uint8).cpu().numpy()
        np.testing.assert_array_equal(got[:, 1:], np.broadcast_to(want[1:], (128, 127)))
