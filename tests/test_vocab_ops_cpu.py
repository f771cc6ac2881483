"""Argument checks of the vocabulary projection and token log-probability calls (CPU only: every call
here is refused, or does nothing, before any CUDA work)."""
import ctypes

import pytest
import torch

from draft_sampling_lossless_markov_gb300 import build, capi
from draft_sampling_lossless_markov_gb300 import torch_api as T

OK, BAD, NO = capi.DSPARK_OK, capi.DSPARK_INVALID_ARG, capi.DSPARK_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    if torch.cuda.is_available():
        pytest.skip("argument-check tests with made-up device addresses: CPU only")
    return capi.load()


def _set(struct, /, **kw):
    for k, v in kw.items():
        setattr(struct, k, v)
    return struct


def _but(struct, /, **kw):
    return _set(type(struct).from_buffer_copy(struct), **kw)


def test_struct_layouts():
    assert ctypes.sizeof(capi.dspark_quant_fp8_args) == 16 + 5 * 8
    assert ctypes.sizeof(capi.dspark_matmul_fp8_args) == 16 + 9 * 8
    assert ctypes.sizeof(capi.dspark_logit_rows) == 24 + 9 * 8
    assert ctypes.sizeof(capi.dspark_token_logprobs_args) == 96 + 8 + 6 * 8
    assert ctypes.sizeof(capi.dspark_token_logprobs_grad_args) == 96 + 8 + 8 * 8


def test_quant_checks():
    a = _set(capi.dspark_quant_fp8_args(), M=4, K=200, dtype=capi.DSPARK_BF16, block_rows=1, x=0x10000, ldx=200,
             codes=0x20000, ldq=208, scale=0x30000)
    for kw in (dict(M=-1), dict(K=0), dict(dtype=5), dict(block_rows=64), dict(x=None), dict(codes=None),
               dict(scale=None), dict(ldx=199), dict(ldq=199), dict(ldx=1 << 50), dict(x=0x10001), dict(scale=0x30002)):
        assert capi.dspark_quant_fp8(_but(a, **kw), 0) == BAD, kw
    assert capi.dspark_quant_fp8(_but(a, M=0, x=None), 0) == OK
    assert capi.load().dspark_quant_fp8(None, None) == BAD


def test_matmul_checks():
    st, n = capi.dspark_matmul_fp8_workspace_size(64, 1000, 200)
    assert st == OK and n >= 256 and n % 256 == 0
    for bad in ((-1, 4, 4), (4, -1, 4), (4, 4, 0)):
        assert capi.dspark_matmul_fp8_workspace_size(*bad)[0] == BAD
    a = _set(capi.dspark_matmul_fp8_args(), M=64, N=1000, K=200, out_dtype=capi.DSPARK_F32, a=0x10000, lda=208,
             a_scale=0x20000, w=0x30000, ldw=208, w_scale=0x40000, out=0x50000, ldo=1000)
    for kw in (dict(M=-1), dict(N=-1), dict(K=0), dict(out_dtype=9), dict(a=None), dict(w=None), dict(a_scale=None),
               dict(w_scale=None), dict(out=None), dict(lda=200), dict(ldw=200), dict(lda=192), dict(a=0x10008),
               dict(w=0x30004), dict(ldo=999), dict(out=0x50002), dict(a_scale=0x20001), dict(w_scale=0x40003)):
        assert capi.dspark_matmul_fp8(_but(a, **kw), 0x100000, n, 0) == BAD, kw
    assert capi.dspark_matmul_fp8(a, 0, n, 0) == BAD
    assert capi.dspark_matmul_fp8(a, 0x100010, n, 0) == BAD
    assert capi.dspark_matmul_fp8(a, 0x100000, 16, 0) == BAD
    assert capi.dspark_matmul_fp8(_but(a, M=0), 0, 0, 0) == OK
    assert capi.dspark_matmul_fp8(_but(a, N=0), 0, 0, 0) == OK


def _rows_cases():
    return (dict(N=-1), dict(V=0), dict(V=capi.DSPARK_MAX_VOCAB + 1), dict(dtype=3), dict(logits=None),
            dict(tokens=None), dict(ld=99), dict(logits=0x10001), dict(mark_req=0x90000), dict(mark_pos=0x90000),
            dict(mark_req=0x90000, mark_pos=0xA0000, n_req=-1), dict(mask=0x70002, mask_ld=4),
            dict(mask=0x70000, mask_ld=3))


def _rows():
    return _set(capi.dspark_logit_rows(), N=8, V=100, dtype=capi.DSPARK_BF16, logits=0x10000, ld=100, tokens=0x60000)


def test_token_logprobs_checks():
    st, n = capi.dspark_token_logprobs_workspace_size(8, 100, 5)
    assert st == OK and n >= 256 and n % 256 == 0
    for bad in ((-1, 10, 0), (1, 0, 0), (1, 10, -1)):
        assert capi.dspark_token_logprobs_workspace_size(*bad)[0] == BAD
    assert capi.dspark_token_logprobs_workspace_size(1, 10, 33)[0] == NO
    a = _set(capi.dspark_token_logprobs_args(), rows=_rows(), top=5, top_id=0x20000, top_logprob=0x30000)
    call = lambda x, ws=0x100000, nb=n: capi.dspark_token_logprobs(x, ws, nb, 0)  # noqa: E731
    for kw in _rows_cases():
        assert call(_but(a, rows=_but(a.rows, **kw))) == BAD, kw
    assert call(_but(a, top=-1)) == BAD and call(_but(a, top=33)) == NO
    assert call(_but(a, top_id=None)) == BAD and call(_but(a, top_logprob=None)) == BAD
    assert call(a, 0) == BAD and call(a, 0x100008) == BAD and call(a, 0x100000, 8) == BAD
    assert call(_but(a, rows=_but(a.rows, N=0)), 0, 0) == OK


def test_token_logprobs_grad_checks():
    a = _set(capi.dspark_token_logprobs_grad_args(), rows=_rows(), top=5, row_stat=0x20000, entropy=0x21000,
             top_id=0x22000, g_logprob=0x23000, g_entropy=0x24000, g_top=0x25000, grad=0x40000, ldg=100)
    call = lambda x, ws=0: capi.dspark_token_logprobs_grad(x, ws, 0)  # noqa: E731
    for kw in _rows_cases():
        assert call(_but(a, rows=_but(a.rows, **kw))) == BAD, kw
    for kw in (dict(row_stat=None), dict(grad=None), dict(entropy=None), dict(top_id=None), dict(g_top=None),
               dict(ldg=99), dict(grad=0x40001), dict(top=-1), dict(grad=0x10000, ldg=128)):
        assert call(_but(a, **kw)) == BAD, kw
    assert call(_but(a, top=33)) == NO
    assert call(a, 0x100008) == BAD
    assert call(_but(a, rows=_but(a.rows, N=0))) == OK


def test_torch_front_end_refuses_host_tensors_and_bad_shapes():
    with pytest.raises(ValueError):
        T.quant_fp8(torch.zeros(2, 4))
    with pytest.raises(ValueError):
        T.matmul_fp8(None, torch.zeros(2, 16, dtype=torch.float8_e4m3fn), torch.zeros(2, 1),
                     torch.zeros(2, 16, dtype=torch.float8_e4m3fn), torch.zeros(1, 1))
    with pytest.raises(TypeError):
        T.token_logprobs(None, torch.zeros(2, 4, dtype=torch.float16), torch.zeros(2, dtype=torch.int32))
