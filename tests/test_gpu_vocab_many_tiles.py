"""matmul_fp8 where every CTA makes several tiles of an output: its rings, buffers and scales go on from tile to
tile.  Codes are whole numbers of at most 8 and scales 1 or 2, so every sum is a whole number below 2^24 (64 * 4 * K,
K <= 4096 here gives at most 2^20): fp32 results are exact, bf16 ones the nearest to the exact value."""
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


def _operands(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M * 31 + N + K)
    kb = -(-K // 128)

    def whole(rows):
        q = T.fp8_codes(rows, K)
        q.copy_(torch.randint(-8, 9, (rows, K), generator=g, device="cuda").to(torch.float8_e4m3fn))
        return q

    def scales(rows):
        return torch.randint(0, 2, (rows, kb), generator=g, device="cuda").float().exp2()

    return whole(M), scales(M), whole(N), scales(-(-N // 128))


def _want(a, sa, w, sw):
    """In fp64 on the GPU; a sample of its columns against the oracle."""
    block = torch.arange(a.shape[1], device="cuda") // 128
    x = a.double() * sa.double()[:, block]
    y = torch.empty((a.shape[0], w.shape[0]), dtype=torch.float64, device="cuda")
    for n in range(0, w.shape[0], 8192):
        rows = torch.arange(n, min(n + 8192, w.shape[0]), device="cuda")
        y[:, n:n + 8192] = x @ (w[n:n + 8192].double() * sw.double()[rows // 128][:, block]).T
    codes = lambda t: t.contiguous().view(torch.uint8).cpu().numpy()  # noqa: E731
    for n in (0, w.shape[0] // 256 * 128, w.shape[0] - 1 - (w.shape[0] - 1) % 128):
        part = w[n:n + 128]
        ref, _ = O.matmul(codes(a), sa.double().cpu().numpy(), codes(part), sw[n // 128:n // 128 + 1].double().cpu().numpy())
        np.testing.assert_array_equal(y[:, n:n + 128].cpu().numpy(), ref)
    return y


def _check(M, N, K, dtype, c0, ld, times=3):
    """A column range from c0 on of rows ld apart; equal calls give equal bits while other work shares the GPU."""
    a, sa, w, sw = _operands(M, N, K)
    want = _want(a, sa, w, sw).to(dtype)
    ws = T.matmul_fp8_workspace(M, N, K)
    store = torch.empty((M, ld), dtype=dtype, device="cuda")
    out = store[:, c0:c0 + N]
    other, side = torch.empty(1 << 26, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(times):
        store.fill_(-7)
        if i:
            with torch.cuda.stream(side):
                other.add_(1)
        T.matmul_fp8(ws, a, sa, w, sw, out=out)
        assert torch.equal(out, want), (i, (out != want).nonzero()[:4].tolist())
        assert bool((store[:, :c0] == -7).all()) and bool((store[:, c0 + N:] == -7).all())
    torch.cuda.synchronize()
    check_no_error(ws)


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("K", [100, 1030, 2560])
@pytest.mark.parametrize("M", [1, 16, 17, 24, 32, 33, 64])
def test_few_rows(M, K, dtype):
    # 2 SMs + 5 tiles of 128 columns: two or three a CTA; rows of an odd length, of 16-byte multiples
    tiles = 2 * _sms() + 5
    _check(M, tiles * 128 - 3, K, dtype, 1, tiles * 128 + 1, times=12 if 16 < M <= 32 else 3)
    _check(M, tiles * 128, K, dtype, 0, tiles * 128, times=1)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,tiles,K", [(1, 24, 2560), (16, 30, 2049), (8, 31, 4096), (3, 60, 1024), (16, 50, 1300),
                                       (16, 61, 1024), (1, 77, 2560), (30, 15, 2560), (30, 36, 1024), (30, 76, 700)])
def test_clusters_over_k(M, tiles, K, dtype):
    # around where the size of the clusters that share a tile's K changes
    _check(M, tiles * 128 - 1, K, dtype, 1, tiles * 128 + 3)


def _pairs():
    return _sms() // 2


@pytest.mark.parametrize("K", [100, 384, 700, 2050])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,wide", [(600, True), (1025, True), (256, True), (300, False), (513, False)])
def test_many_rows(M, wide, K, dtype):
    # two tiles or more a CTA pair, of 256 columns (where tiles are many) and of 128 (some 2.1 a pair); the last ones ragged
    row_tiles = -(-M // 256)
    n256 = -(-(2 * _pairs() + 5) // row_tiles) if wide else 0
    N = n256 * 256 + 129 if wide else -(-(2 * _pairs() + 3) // row_tiles) * 128 - 41
    _check(M, N, K, dtype, 1, N + 2)  # rows that TMA cannot store
    ld = -(-N // 16) * 16
    _check(M, N, K, dtype, 0, ld, times=2)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(2048, 12288, 512), (777, 30011, 1030)])
def test_many_tiles_a_pair(M, N, K, dtype):
    _check(M, N, K, dtype, 0, -(-N // 16) * 16, times=2)


@pytest.mark.parametrize("M,count", [(64, 20), (64, 64), (32, 1), (600, 300), (600, 599), (2048, 60), (2048, 0)])
def test_row_count_on_the_device(M, count):
    K, N = 700, (2 * _sms() + 5) * 128 - 3
    a, sa, w, sw = _operands(M, N, K)
    want = _want(a[:max(count, 1)], sa[:max(count, 1)], w, sw)[:count]
    ws = T.matmul_fp8_workspace(M, N, K)
    n = torch.tensor([count], dtype=torch.int32, device="cuda")
    for dtype, ld in ((BF16, N + 3), (F32, N + 2), (F32, N)):
        store = torch.full((M, ld), -7.0, dtype=dtype, device="cuda")
        T.matmul_fp8(ws, a, sa, w, sw, out=store[:, :N], n_rows=n)
        assert torch.equal(store[:count, :N], want.to(dtype))
        assert bool((store[count:] == -7).all()) and bool((store[:, N:] == -7).all())
    check_no_error(ws)
