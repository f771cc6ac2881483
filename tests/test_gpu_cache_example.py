"""The example with an attention layer: its steps run, its attention is the oracle's over the cache that they wrote, and a
tree's path stays in it."""
import numpy as np
import pytest
import torch

from examples import decode_with_cache as E
from gpu_common import check_no_error, require_gpu
from kv_common import as_numpy, bits, i32, np64
from oracle import kv_cache as O
from draft_sampling_lossless_markov_gb300 import torch_api as T

pytestmark = pytest.mark.gpu

NORM = 0.004  # as in the attention's own tests


def test_steps():
    require_gpu()
    s = E.make()
    B, total = E.WORKLOAD.B, s["base"].clone()
    for _ in range(3):
        r = E.step(s)
        off, base = r["schedule"]["offsets"].tolist(), r["base"].tolist()
        n = off[-1]
        assert n == int(r["schedule"]["n_verify"][0])
        want = O.attention(as_numpy(s["cache"]), np64(r["q"][:n]), off, base, E.D ** -0.5)
        got = np64(s["attended"][:n])
        assert np.linalg.norm(got - want) < NORM * np.linalg.norm(want)
        total += r["verify"]["n_out"]
        assert (r["verify"]["n_out"] >= 1).all() and torch.equal(total, s["base"])
    for ws in s.values():
        if isinstance(ws, T.Workspace):
            check_no_error(ws)
    # nodes 1 and 3 of four drafted rows become the context's next two
    place = i32(np.repeat(np.arange(B), 4)), i32(np.tile(np.arange(4), B))
    k, v = T.cache_read(s["cache"], *place, base=s["base"])
    E.keep_path(s, s["base"], i32(np.tile([1, 3], (B, 1))), i32(np.full(B, 2)))
    k2, v2 = T.cache_read(s["cache"], *place, base=s["base"])
    for a, b in ((k, k2), (v, v2)):
        a, b = (t.view(B, 4, E.HKV, E.D) for t in (a, b))
        assert torch.equal(bits(b[:, 0]), bits(a[:, 1])) and torch.equal(bits(b[:, 1]), bits(a[:, 3]))
        assert torch.equal(bits(b[:, 2:]), bits(a[:, 2:]))


def test_main(capsys):
    require_gpu()
    E.main()
    assert "context lengths" in capsys.readouterr().out
