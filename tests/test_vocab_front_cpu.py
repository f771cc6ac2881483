"""The front end's packed structs are the C structs, and sizes above 2^30 are refused (no GPU needed)."""
import ctypes

import pytest

from draft_sampling_lossless_markov_gb300 import capi


def _fill(kind, values):
    s = kind()
    for name, t in kind._fields_:
        if issubclass(t, ctypes.Structure):
            setattr(s, name, _fill(t, values))
        else:
            setattr(s, name, values.pop(0))
    return s


def _count(kind):
    return sum(_count(t) if issubclass(t, ctypes.Structure) else 1 for _, t in kind._fields_)


@pytest.mark.parametrize("name", ["quant_fp8", "matmul_fp8", "token_logprobs", "token_logprobs_grad"])
def test_packed_structs_are_the_c_structs(name):
    kind = getattr(capi, f"dspark_{name}_args")
    values = [3 + 7 * i for i in range(_count(kind))]
    packed = getattr(capi, f"pack_{name}")(*values)
    s = _fill(kind, list(values))
    again = kind.from_buffer_copy(packed)

    def same(a, b):
        for n, t in a._fields_:
            x, y = getattr(a, n), getattr(b, n)
            assert same(x, y) if issubclass(t, ctypes.Structure) else x == y, n
        return True

    assert len(packed) == ctypes.sizeof(kind) and same(s, again)


@pytest.mark.parametrize("M,N,K", [(2 ** 30 + 1, 8, 16), (8, 2 ** 30 + 1, 16), (8, 8, 2 ** 30 + 16)])
def test_huge_sizes_are_refused(M, N, K):
    at = 1 << 20  # an address that is never read: the refusal comes first
    a = capi.pack_matmul_fp8(M, N, K, capi.DSPARK_F32, at, K + (-K) % 16, at, at, K + (-K) % 16, at, at, N, 0)
    assert capi.dspark_matmul_fp8(a, at, 1 << 30, 0) == capi.DSPARK_UNSUPPORTED
    if N == 8:
        q = capi.pack_quant_fp8(M, K, capi.DSPARK_BF16, 1, at, K, at, K, at)
        assert capi.dspark_quant_fp8(q, 0) == capi.DSPARK_UNSUPPORTED
