"""A process whose first call of each form of the vocabulary operators is the one a stream capture records: the replay
gives the bits of a plain call after it."""
import os
import subprocess
import sys

import pytest

from gpu_common import require_gpu

pytestmark = pytest.mark.gpu

PROGRAM = """
import torch
from draft_sampling_lossless_markov_gb300 import torch_api as T
BF16, F32 = torch.bfloat16, torch.float32
g = torch.Generator(device="cuda").manual_seed(1)
rand = lambda *s: torch.randn(s, generator=g, device="cuda")

def check(call, outs):
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for t in outs:
        t.zero_()
    graph.replay()
    first = [t.clone() for t in outs]
    for t in outs:
        t.zero_()
    call()
    torch.cuda.synchronize()
    for a, b in zip(first, outs):
        assert torch.equal(a.view(torch.uint8), b.contiguous().view(torch.uint8))

for dt in (BF16, F32):
    for rows in (1, 128):
        for M, K in ((40, 256), (40, 255), (8192, 4096 + 8)):
            x = rand(M, K).to(dt)
            codes = torch.empty((M, K), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
            scale = torch.empty((-(-M // rows), -(-K // 128)), device="cuda")
            check(lambda: T.quant_fp8(x, rows, out=(codes, scale)), (codes.view(torch.uint8), scale))
ws = T.matmul_fp8_workspace(1500, 40001, 512)
for dt in (BF16, F32):
    for M in (9, 20, 40, 300, 1500):
        for N in (300, 40001):
            a, w = T.fp8_codes(M, 512), T.fp8_codes(N, 512)
            a.copy_(rand(M, 512).to(torch.float8_e4m3fn)), w.copy_(rand(N, 512).to(torch.float8_e4m3fn))
            sa, sw = torch.ones((M, 4), device="cuda"), torch.ones((-(-N // 128), 4), device="cuda")
            out = torch.empty((M, N), dtype=dt, device="cuda")
            check(lambda: T.matmul_fp8(ws, a, sa, w, sw, out=out), (out,))
lw = T.token_logprobs_workspace(700, 50000, 5)
for dt in (BF16, F32):
    for N, V in ((1, 50000), (700, 5000), (300, 50000)):
        z, tok = rand(N, V).to(dt), torch.arange(N, dtype=torch.int32, device="cuda")
        for mask in (None, torch.full((N, -(-V // 32)), -2, dtype=torch.int32, device="cuda")):
            for top in (0, 5):
                o = dict(logprob=torch.empty(N, device="cuda"), row_stat=torch.empty((N, 2), device="cuda"),
                         top_id=torch.empty((N, top), dtype=torch.int32, device="cuda"),
                         top_logprob=torch.empty((N, top), device="cuda"))
                check(lambda: T.token_logprobs(lw, z, tok, top=top, mask=mask, out=o), tuple(o.values()))
        d = torch.empty_like(z)
        check(lambda: T.token_logprobs_grad(lw, z, tok, o["row_stat"], g_logprob=o["logprob"], out=d), (d,))
for w in (ws, lw):
    assert w.read_error()[0] == 0
print("done")
"""


def test_first_calls_under_capture():
    require_gpu()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("done\n"), r.stdout + r.stderr
