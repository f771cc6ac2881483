"""Row counts and workspace sizes above 2^30 are refused by every vocabulary call (no GPU needed; the made-up
addresses are never read)."""
import pytest
import torch

from draft_sampling_lossless_markov_gb300 import build, capi

NO, BAD = capi.DSPARK_UNSUPPORTED, capi.DSPARK_INVALID_ARG
HUGE, AT = 2 ** 30 + 1, 1 << 20


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    if torch.cuda.is_available():
        pytest.skip("made-up device addresses: CPU only")


def _rows(N, V=2):
    return N, V, capi.DSPARK_F32, 0, 0, AT, V, AT, 0, 0, 0, 0, 0, 0


def test_row_calls():
    a = capi.pack_token_logprobs(*_rows(HUGE), 0, AT, AT, AT, AT, 0, 0)
    assert capi.dspark_token_logprobs(a, AT, 1 << 20, 0) == NO
    g = capi.pack_token_logprobs_grad(*_rows(HUGE), 0, AT, 0, 0, AT, 0, 0, AT + 4096, 2)
    assert capi.dspark_token_logprobs_grad(g, 0, 0) == NO
    # what is wrong is reported before what is too large
    a = capi.pack_token_logprobs(*_rows(HUGE, capi.DSPARK_MAX_VOCAB + 1), 0, AT, AT, AT, AT, 0, 0)
    assert capi.dspark_token_logprobs(a, AT, 1 << 20, 0) == BAD


def test_workspace_sizes():
    assert capi.dspark_token_logprobs_workspace_size(HUGE, 2, 0)[0] == NO
    assert capi.dspark_token_logprobs_workspace_size(2 ** 30, 2, 0)[0] == capi.DSPARK_OK
    for sizes in ((HUGE, 8, 16), (8, HUGE, 16), (8, 8, HUGE)):
        assert capi.dspark_matmul_fp8_workspace_size(*sizes)[0] == NO
