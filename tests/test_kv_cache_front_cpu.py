"""What the torch front end of the cache refuses, without a GPU."""
import pytest
import torch

from draft_sampling_lossless_markov_gb300 import torch_api as T


@pytest.mark.parametrize("name", ["table", "k", "v", "k_scale", "v_scale", "n_req", "fields"])
def test_a_cache_keeps_its_tensors(name, monkeypatch):
    """Another tensor in the place of one whose address the calls have taken."""
    monkeypatch.setattr(T, "_rows", lambda t, *a: (t.data_ptr(), t.stride(0), *t.shape))
    monkeypatch.setattr(T, "_dense", lambda t, *a: None if t is None else t.data_ptr())
    pool = [torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16) for _ in range(2)]
    table = torch.zeros((1, 2), dtype=torch.int32)
    c = T.KvCache(*pool, table)
    with pytest.raises(AttributeError, match="keeps its tensors"):
        setattr(c, name, table.clone())
    assert c.table is table and c.k is pool[0] and c.fields[7:9] == tuple(t.data_ptr() for t in pool)
    c.table[0, 1] = 1  # in place
