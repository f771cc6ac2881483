"""The vocabulary operators on buffers of more than 2^31 elements: the last rows, whose offsets pass 32 bits, are those of
the same call on these rows alone (equal bits where the call's form is the same; whole numbers for the product)."""
import pytest
import torch

from draft_sampling_lossless_markov_gb300 import torch_api as T
from gpu_common import check_no_error, require_gpu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def _fill(t, scale, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    for i in range(0, t.shape[0], 4096):
        part = t[i:i + 4096]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * scale)
    return t


def _bytes(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quant(block_rows):
    M, K = 2200 * 1024, 1030  # 2.3e9 elements; rows of 1030 elements are read unaligned
    x = _fill(torch.empty((M, K), dtype=BF16, device="cuda"), 3.0)
    codes, scale = T.quant_fp8(x, block_rows)
    for lo in (0, M // 2, M - 256):
        c, s = T.quant_fp8(x[lo:lo + 256].clone(), block_rows)
        assert torch.equal(_bytes(codes[lo:lo + 256]), _bytes(c))
        assert torch.equal(scale[lo // block_rows:(lo + 256) // block_rows], s)


def _whole(rows, K, seed):
    q = T.fp8_codes(rows, K)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for i in range(0, rows, 65536):
        n = min(65536, rows - i)
        q[i:i + n] = torch.randint(-8, 9, (n, K), generator=g, device="cuda").to(torch.float8_e4m3fn)
    return q


@pytest.mark.parametrize("M,N,K,ld", [(17000, 131072, 144, 131072), (17000, 131071, 144, 131073), (1, 1100000, 2048, 1100000),
                                      (24, 1100000, 2048, 1100001), (300, 7200000, 144, 7200000)])
def test_product(M, N, K, ld):
    a, w = _whole(M, K, 1), _whole(N, K, 2)
    kb = -(-K // 128)
    sa, sw = torch.ones((M, kb), device="cuda"), torch.ones((-(-N // 128), kb), device="cuda")
    store = torch.full((M, ld), -7.0, dtype=BF16, device="cuda")
    ws = T.matmul_fp8_workspace(M, N, K)
    T.matmul_fp8(ws, a, sa, w, sw, out=store[:, :N])
    check_no_error(ws)
    for r in (slice(0, 64), slice(max(0, M - 300), M)):
        for c in (slice(0, 200), slice(N // 2, N // 2 + 200), slice(N - 200, N)):
            want = (a[r].double() @ w[c].double().T).to(BF16)
            assert torch.equal(store[r, c], want)
    assert bool((store[:, N:] == -7).all())


@pytest.mark.parametrize("masked", [False, True])
def test_answers_and_gradient(masked):
    N, V = 15000, 151936
    z = _fill(torch.empty((N, V), dtype=BF16, device="cuda"), 3.0)
    tok = (torch.arange(N, device="cuda") * 9973 % V).to(torch.int32)
    mask = torch.randint(-2 ** 31, 2 ** 31, (N, V // 32), device="cuda").to(torch.int32) if masked else None
    ws = T.token_logprobs_workspace(N, V, 6)
    out = T.token_logprobs(ws, z, tok, top=6, mask=mask)
    n = 2048  # enough rows for the same form of the kernel
    rows = slice(N - n, N)
    few = T.token_logprobs(ws, z[rows].clone(), tok[rows], top=6, mask=None if mask is None else mask[rows].clone())
    for k in out:
        assert torch.equal(out[k][rows], few[k]), k
    g = torch.linspace(-1, 1, N, device="cuda")
    want = T.token_logprobs_grad(ws, z[rows].clone(), tok[rows], few["row_stat"], g_logprob=g[rows].clone(),
                                 mask=None if mask is None else mask[rows].clone())
    T.token_logprobs_grad(ws, z, tok, out["row_stat"], g_logprob=g, mask=mask, out=z)
    check_no_error(ws)
    assert torch.equal(z[rows], want)
