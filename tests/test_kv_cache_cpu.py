"""Argument checks of the cache and tree attention calls (CPU only: every call here is refused, or does nothing, before any
CUDA work), their structs, and pins of their oracle."""
import ctypes

import numpy as np
import pytest
import torch

from draft_sampling_lossless_markov_gb300 import build, capi
from draft_sampling_lossless_markov_gb300 import torch_api as T
from oracle import kv_cache as O

OK, BAD, NO = capi.DSPARK_OK, capi.DSPARK_INVALID_ARG, capi.DSPARK_UNSUPPORTED


@pytest.fixture(scope="module")
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


def _cache():
    return _set(capi.dspark_kv_cache(), n_pages=10, page_size=16, n_kv_heads=2, head_dim=64, dtype=capi.DSPARK_E4M3, n_req=3,
                max_pages=4, k=0x10000, v=0x20000, k_scale=0x30000, v_scale=0x40000, table=0x50000, table_ld=4)


CACHE_CASES = [(dict(n_pages=0), BAD), (dict(n_kv_heads=0), BAD), (dict(n_req=-1), BAD), (dict(max_pages=0), BAD),
               (dict(page_size=0), BAD), (dict(page_size=24), BAD), (dict(page_size=-16), BAD), (dict(dtype=1), BAD), (dict(dtype=3), BAD),
               (dict(head_dim=0), BAD), (dict(page_size=8), NO), (dict(page_size=2048), NO), (dict(head_dim=80), NO),
               (dict(head_dim=256), NO), (dict(n_pages=1 << 26), NO), (dict(n_kv_heads=1 << 23), NO),
               (dict(max_pages=1 << 27, table_ld=1 << 27), NO), (dict(k=None), BAD), (dict(v=None), BAD), (dict(k=0x10008), BAD),
               (dict(v=0x20004), BAD), (dict(k_scale=None), BAD), (dict(v_scale=None), BAD), (dict(k_scale=0x30008), BAD),
               (dict(v_scale=0x40004), BAD), (dict(table=None), BAD), (dict(table=0x50002), BAD), (dict(table_ld=3), BAD)]


def _rows(kind):
    return _set(kind(), cache=_cache(), N=5, dtype=capi.DSPARK_BF16, k=0x60000, ldk=128, v=0x70000, ldv=128, mark_req=0x80000,
                mark_pos=0x90000)


@pytest.mark.parametrize("name", ["write", "read"])
def test_write_and_read_checks(lib, name):
    a = _rows(getattr(capi, f"dspark_cache_{name}_args"))
    f = getattr(capi, f"dspark_cache_{name}")
    for kw, st in CACHE_CASES:
        assert f(_but(a, cache=_but(a.cache, **kw)), 0, 0) == st, kw
    for kw in (dict(N=-1), dict(dtype=2), dict(dtype=-1), dict(k=None), dict(v=None), dict(k=0x60008), dict(v=0x70002),
               dict(ldk=127), dict(ldk=132), dict(ldv=120), dict(ldv=1 << 50), dict(mark_req=None), dict(mark_pos=None)):
        assert f(_but(a, **kw), 0, 0) == BAD, kw
    assert f(a, 0x100010, 0) == BAD
    assert f(_but(a, N=(1 << 30) + 1), 0, 0) == NO
    assert f(_but(a, N=0, k=None, mark_req=None), 0, 0) == OK
    assert getattr(lib, f"dspark_cache_{name}")(None, None, None) == BAD


def test_move_checks(lib):
    a = _set(capi.dspark_cache_move_args(), cache=_cache(), path_cols=4, base=0x60000, path=0x70000, path_ld=4, n_path=0x80000)
    for kw, st in CACHE_CASES:
        assert capi.dspark_cache_move(_but(a, cache=_but(a.cache, **kw)), 0, 0) == st, kw
    for kw, st in ((dict(path_cols=0), BAD), (dict(path_cols=65), NO), (dict(base=None), BAD), (dict(path=None), BAD),
                   (dict(n_path=None), BAD), (dict(path_ld=3), BAD)):
        assert capi.dspark_cache_move(_but(a, **kw), 0, 0) == st, kw
    assert capi.dspark_cache_move(a, 0x100008, 0) == BAD
    assert capi.dspark_cache_move(_but(a, cache=_but(a.cache, n_req=0, table=None)), 0, 0) == OK
    assert lib.dspark_cache_move(None, None, None) == BAD


def test_attention_checks(lib):
    st, n = capi.dspark_tree_attention_workspace_size(3, 8, 8, 2, 64)
    assert st == OK and n >= 256 and n % 256 == 0
    for sizes, st in (((-1, 8, 8, 2, 64), BAD), ((3, 0, 8, 2, 64), BAD), ((3, 65, 8, 2, 64), NO), ((3, 8, 0, 2, 64), BAD),
                      ((3, 8, 7, 2, 64), BAD), ((3, 8, 8, 0, 64), BAD), ((3, 8, 8, 2, 0), BAD), ((3, 8, 8, 2, 96), NO),
                      ((3, 8, 1 << 17, 2, 64), NO), (((1 << 30) + 1, 8, 8, 2, 64), NO)):
        assert capi.dspark_tree_attention_workspace_size(*sizes)[0] == st, sizes
    assert lib.dspark_tree_attention_workspace_size(3, 8, 8, 2, 64, None) == BAD
    a = _set(capi.dspark_tree_attention_args(), cache=_cache(), N=20, n_q_heads=8, max_tree=8, scale=0.1, q=0x60000, ldq=512,
             out=0x70000, ldo=512, offsets=0x80000, base=0x90000)
    call = lambda x, ws=0x100000, nb=n: capi.dspark_tree_attention(x, ws, nb, 0)  # noqa: E731
    for kw, st in CACHE_CASES:
        if kw != dict(n_kv_heads=1 << 23):  # 8 query heads are no multiple of it
            assert call(_but(a, cache=_but(a.cache, **kw))) == st, kw
    for kw, st in ((dict(N=-1), BAD), (dict(n_q_heads=0), BAD), (dict(n_q_heads=7), BAD), (dict(max_tree=0), BAD),
                   (dict(max_tree=65), NO), (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(q=None), BAD),
                   (dict(out=None), BAD), (dict(q=0x60008), BAD), (dict(out=0x70002), BAD), (dict(ldq=511), BAD),
                   (dict(ldq=516), BAD), (dict(ldo=504), BAD), (dict(offsets=None), BAD), (dict(base=None), BAD),
                   (dict(tree=0xA0004), BAD), (dict(N=(1 << 30) + 1), NO)):
        assert call(_but(a, **kw)) == st, kw
    assert call(a, 0) == BAD and call(a, 0x100008) == BAD and call(a, 0x100000, n - 256) == BAD
    assert call(_but(a, N=0, q=None), 0, 0) == OK
    assert call(_but(a, cache=_but(a.cache, n_req=0, table=None)), 0, 0) == OK


def test_addresses_and_sizes_beyond_the_kernels(lib):
    """Integers that do not begin on 4 bytes, and more query heads a kv head than columns can be told apart for."""
    for name in ("write", "read"):
        a = _rows(getattr(capi, f"dspark_cache_{name}_args"))
        for kw in (dict(mark_req=0x80002), dict(mark_pos=0x90001), dict(base=0xA0002), dict(n_rows=0xB0003)):
            assert getattr(capi, f"dspark_cache_{name}")(_but(a, **kw), 0, 0) == BAD, kw
    a = _set(capi.dspark_cache_move_args(), cache=_cache(), path_cols=4, base=0x60000, path=0x70000, path_ld=4, n_path=0x80000)
    for kw in (dict(base=0x60002), dict(path=0x70001), dict(n_path=0x80002)):
        assert capi.dspark_cache_move(_but(a, **kw), 0, 0) == BAD, kw
    n = capi.dspark_tree_attention_workspace_size(3, 8, 8, 2, 64)[1]
    a = _set(capi.dspark_tree_attention_args(), cache=_cache(), N=20, n_q_heads=8, max_tree=8, scale=0.1, q=0x60000, ldq=512,
             out=0x70000, ldo=512, offsets=0x80000, base=0x90000)
    for kw in (dict(offsets=0x80002), dict(base=0x90001)):
        assert capi.dspark_tree_attention(_but(a, **kw), 0x100000, n, 0) == BAD, kw
    size = capi.dspark_tree_attention_workspace_size
    assert size(3, 64, 4096, 1, 64)[0] == OK and size(3, 64, 1 << 16, 16, 64)[0] == OK
    assert size(3, 1, 4097, 1, 64)[0] == NO and size(3, 1, (1 << 16) + 16, 16, 64)[0] == NO
    for group in (1, 3, 7, 100, 4095, 4096):  # a column over the group, as the kernel forms it
        inv, c = ((1 << 32) + group - 1) // group, np.arange(64 * group + 64, dtype=np.uint64)
        np.testing.assert_array_equal(c * np.uint64(inv) >> np.uint64(32), c // np.uint64(group))


def test_packed_structs_are_the_c_structs():
    for name in ("cache_write", "cache_read", "cache_move", "tree_attention"):
        kind = getattr(capi, f"dspark_{name}_args")
        fields = [t for _, t in capi.dspark_kv_cache._fields_] + [t for _, t in kind._fields_[1:]]
        values = [0.5 + i if t is ctypes.c_float else 3 + 7 * i for i, t in enumerate(fields)]
        s = kind.from_buffer_copy(getattr(capi, f"pack_{name}")(*values))
        got = [getattr(s.cache, n) for n, _ in capi.dspark_kv_cache._fields_] + [getattr(s, n) for n, _ in kind._fields_[1:]]
        assert got == values and len(bytes(s)) == ctypes.sizeof(kind)


def test_front_end_refuses():
    z = torch.zeros
    f8 = torch.float8_e4m3fn
    with pytest.raises(ValueError):  # host tensors
        T.KvCache(z(2, 1, 16, 64, dtype=torch.bfloat16), z(2, 1, 16, 64, dtype=torch.bfloat16), z(1, 2, dtype=torch.int32))
    with pytest.raises(TypeError):
        T.KvCache(z(2, 1, 16, 64), z(2, 1, 16, 64), z(1, 2, dtype=torch.int32))
    with pytest.raises(ValueError):  # codes without scales, scales without codes, too few dimensions
        T.KvCache(z(2, 1, 16, 64, dtype=torch.uint8).view(f8), z(2, 1, 16, 64, dtype=torch.uint8).view(f8), z(1, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        T.KvCache(z(2, 1, 16, 64, dtype=torch.bfloat16), z(2, 1, 16, 64, dtype=torch.bfloat16), z(1, 2, dtype=torch.int32),
                  z(2, 1, 16), z(2, 1, 16))
    with pytest.raises(ValueError):
        T.KvCache(z(2, 16, 64, dtype=torch.bfloat16), z(2, 16, 64, dtype=torch.bfloat16), z(1, 2, dtype=torch.int32))


# --------------------------------------------------------------------------- the oracle against hand-worked values
def _small(scales=False):
    k = np.arange(3 * 1 * 2 * 2, dtype=np.float64).reshape(3, 1, 2, 2)
    s = np.full((3, 1, 2), 2.0) if scales else None
    return dict(k=k.copy(), v=-k, k_scale=s, v_scale=s, table=np.array([[2, 0], [1, -1]]))


def test_oracle_places_and_moves():
    c = _small()
    assert O.place(c, 0, 0) == (2, 0) and O.place(c, 0, 3) == (0, 1) and O.place(c, 1, 2) is None and O.place(c, 0, 4) is None
    np.testing.assert_array_equal(O.rows(_small(True), "k", 0, [1, 2])[:, 0], [[20, 22], [0, 2]])
    O.move(c, [0, 0], np.array([[0, 2, 1], [1, 0, 9]]), [3, 2])  # request 0: 1 <- 2, 2 <- 1; request 1 swaps
    np.testing.assert_array_equal(c["k"][2, 0], [[8, 9], [0, 1]])
    np.testing.assert_array_equal(c["k"][0, 0], [[10, 11], [2, 3]])
    np.testing.assert_array_equal(c["k"][1, 0], [[6, 7], [4, 5]])


def test_oracle_attention():
    c = _small()
    q = np.zeros((3, 2, 2))
    # equal scores: the mean of what is seen; row 0 of request 0 sees positions 0, 1 and itself
    out = O.attention(c, q, [0, 2, 3], [2, 0], 1.0)
    np.testing.assert_allclose(out[0, 0], -np.array([8 + 10 + 0, 9 + 11 + 1]) / 3)
    np.testing.assert_allclose(out[1, 1], -np.array([8 + 10 + 0 + 2, 9 + 11 + 1 + 3]) / 4)
    np.testing.assert_allclose(out[2, 0], [-4, -5])
    tree = np.array([1, 2, 0], dtype=np.uint64)
    out = O.attention(c, q, [0, 2, 3], [2, 0], 1.0, tree)
    np.testing.assert_allclose(out[1, 0], -np.array([8 + 10 + 2, 9 + 11 + 3]) / 3)
    np.testing.assert_array_equal(out[2], 0.0)
    q[0, 0] = [1.0, 0.0]
    p = np.exp([8.0, 10.0, 0.0])
    np.testing.assert_allclose(O.attention(c, q, [0, 2, 3], [2, 0], 1.0)[0, 0], -(p / p.sum()) @ np.array([[8, 9], [10, 11], [0, 1]]))
    np.testing.assert_allclose(O.attention(c, 2 * q, [0, 2, 3], [2, 0], 0.5)[0, 0], -(p / p.sum()) @ np.array([[8, 9], [10, 11], [0, 1]]))


def test_oracle_write_rounds_to_the_nearest_code():
    c = _small(True)
    x = np.array([[[448.0, 17.1]], [[0.0, 0.0]]])
    assert O.write(c, x, x, [0, 1], [1, 0], [0, 0], 2) == []
    np.testing.assert_array_equal(c["k"][2, 0, 1], [448, 18])  # steps of 2 between 16 and 32
    assert c["k_scale"][2, 0, 1] == 1.0 and c["k_scale"][1, 0, 0] == 2.0 ** -100 / 448
    assert O.write(c, x, x, [1, 3], [2, 0], [0, 0], 2) == [0, 1]
