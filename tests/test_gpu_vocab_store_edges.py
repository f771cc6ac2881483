"""matmul_fp8 into a column range of a wider buffer whose rows are 16-byte aligned: nothing beside the range is written,
whatever the range's length is a multiple of.  Operands are whole numbers, so results are exact."""
import pytest
import torch

from draft_sampling_lossless_markov_gb300 import torch_api as T
from gpu_common import check_no_error, require_gpu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("M", [1, 40, 65, 150, 600])
@pytest.mark.parametrize("N", [1, 3, 31, 32, 33, 127, 260, 261, 262, 515, 1000, 1031, 8195, 13697])
def test_columns_beside_the_output_stay(M, N):
    K = 200
    g = torch.Generator(device="cuda").manual_seed(M + N)

    def whole(rows):
        q = T.fp8_codes(rows, K)
        q.copy_(torch.randint(-8, 9, (rows, K), generator=g, device="cuda").to(torch.float8_e4m3fn))
        return q

    a, w = whole(M), whole(N)
    sa, sw = torch.ones((M, 2), device="cuda"), torch.ones((-(-N // 128), 2), device="cuda")
    want = a.double() @ w.double().T
    ws = T.matmul_fp8_workspace(M, N, K)
    for dtype in (BF16, F32):
        for c0 in (0, 8):
            store = torch.full((M + 1, c0 + -(-N // 16) * 16 + 16), -7.0, dtype=dtype, device="cuda")
            T.matmul_fp8(ws, a, sa, w, sw, out=store[:M, c0:c0 + N])
            assert torch.equal(store[:M, c0:c0 + N], want.to(dtype))
            assert bool((store[:M, :c0] == -7).all()) and bool((store[:M, c0 + N:] == -7).all())
            assert bool((store[M] == -7).all())
    check_no_error(ws)
