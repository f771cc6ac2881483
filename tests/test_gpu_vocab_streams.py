"""Calls of every form on several streams at once give the bits of the same calls alone (each stream with its own
workspace, as the calls ask)."""
import random

import pytest
import torch

from draft_sampling_lossless_markov_gb300 import torch_api as T
from gpu_common import check_no_error, require_gpu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _calls():
    """(function of (workspaces, stream) that returns its outputs, ...)"""
    g = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    calls = []
    for M, N, K, dt in ((1, 2560, 2560, BF16), (8, 2560, 2560, BF16), (16, 30000, 512, F32), (20, 1900, 2560, BF16),
                        (30, 25000, 384, BF16), (64, 1900, 2560, F32), (64, 21000, 640, BF16), (300, 5000, 384, BF16),
                        (700, 4099, 1030, F32), (1000, 12000, 256, BF16)):
        a, sa = T.quant_fp8(rand(M, K))
        w, sw = T.quant_fp8(rand(N, K), 128)
        calls.append(lambda ws, s, a=a, sa=sa, w=w, sw=sw, dt=dt: (T.matmul_fp8(ws[0], a, sa, w, sw, out_dtype=dt, stream=s),))
    for N, V, dt, top in ((1, 151936, BF16, 20), (9, 30001, F32, 0), (300, 5000, BF16, 8), (700, 9000, BF16, 3)):
        z, tok = rand(N, V).to(dt), torch.arange(N, device="cuda", dtype=torch.int32)
        calls.append(lambda ws, s, z=z, tok=tok, top=top: tuple(T.token_logprobs(ws[1], z, tok, top=top, stream=s).values()))
        f = T.token_logprobs(T.token_logprobs_workspace(N, V, top), z, tok, top=top)
        calls.append(lambda ws, s, z=z, tok=tok, f=f: (T.token_logprobs_grad(ws[1], z, tok, f["row_stat"], g_logprob=f["logprob"],
                                                                             stream=s),))
    for M, K, rows in ((64, 4096, 1), (2000, 2050, 1), (1000, 1000, 128)):
        x = rand(M, K).to(BF16)
        calls.append(lambda ws, s, x=x, rows=rows: T.quant_fp8(x, rows, stream=s))
    return calls


def test_streams_at_once():
    require_gpu()
    calls = _calls()
    new = lambda: (T.matmul_fp8_workspace(1, 1, 1), T.token_logprobs_workspace(1, 1, 1))  # noqa: E731
    alone = new()
    want = []
    for c in calls:
        want.append([t.clone() for t in c(alone, None)])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    spaces = [new() for _ in streams]
    torch.cuda.synchronize()
    rng = random.Random(3)
    for _ in range(12):
        got = []
        for _ in range(60):
            k, i = rng.randrange(len(calls)), rng.randrange(len(streams))
            with torch.cuda.stream(streams[i]):
                got.append((k, calls[k](spaces[i], streams[i])))
        torch.cuda.synchronize()
        for k, outs in got:
            for a, b in zip(outs, want[k]):
                assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), k
    for ws in spaces:
        check_no_error(ws[0])
        check_no_error(ws[1])
