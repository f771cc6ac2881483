"""The cache calls on rows of more than 2^31 elements: the last heads lie past what 32 bits can count."""
import numpy as np
import pytest
import torch

from draft_sampling_lossless_markov_gb300 import torch_api as T
from gpu_common import require_gpu
from kv_common import BF16, E4M3, bits, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
def test_rows_past_32_bits(D):
    require_gpu()
    torch.cuda.empty_cache()
    heads, page = (1 << 31) // D + 40, 16
    if torch.cuda.mem_get_info()[0] < 110 << 30:
        pytest.skip("needs 110 GB")
    pools = [torch.empty((1, heads, page, D), dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    scales = [torch.empty((1, heads, page), device="cuda") for _ in range(2)]
    c = T.KvCache(*pools, i32([[0]]), *scales)
    x = torch.empty((1, heads, D), dtype=BF16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(D))
    T.cache_write(c, x, x, i32([0]), i32([3]))
    back = T.cache_read(c, i32([0]), i32([3]))
    T.cache_move(c, i32([0]), i32([[3]]), i32([1]))
    moved = T.cache_read(c, i32([0]), i32([0]))
    assert all(torch.equal(a, b) for a, b in zip(back, moved)) and torch.equal(*back)
    small = T.KvCache.create(1, page, 40, D, i32([[0]]))
    for lo in (0, heads // 2, (1 << 31) // D - 20, heads - 40):
        part = x[:, lo:lo + 40].contiguous()
        T.cache_write(small, part, part, i32([0]), i32([3]))
        for a, b in zip((*pools, *scales), (small.k, small.v, small.k_scale, small.v_scale)):
            assert np.array_equal(bits(a[:, lo:lo + 40, 3]).cpu().numpy(), bits(b[:, :, 3]).cpu().numpy())
        want = T.cache_read(small, i32([0]), i32([3]))
        assert all(torch.equal(a[:, lo:lo + 40], b) for a, b in zip(back, want))
    del pools, scales, c, x, back, moved
    torch.cuda.empty_cache()
