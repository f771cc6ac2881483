"""The vocabulary operators may be set up while the kernels before them in their stream drain.  Chains of calls
without a wait in between, over buffers that the next step overwrites, give the bits of the same calls made
one at a time."""
import pytest
import torch

from draft_sampling_lossless_markov_gb300 import torch_api as T
from examples import verify_with_answers as E
from gpu_common import check_no_error, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _chain(xs, w, w_scale, tokens, wait):
    """Per step: quantise, project, answer, gradient.  Codes, logits and statistics are the next step's too."""
    (n, M, K), V, top = xs.shape, w.shape[0], 4
    wait()
    ws, lw = T.matmul_fp8_workspace(M, V, K), T.token_logprobs_workspace(M, V, top)
    codes, scale = T.fp8_codes(M, K), torch.empty((M, -(-K // 128)), device="cuda")
    logits = torch.empty((M, V), dtype=torch.bfloat16, device="cuda")
    stat = torch.empty((M, 2), device="cuda")
    weight = torch.linspace(-1, 1, M, device="cuda")
    lp = torch.zeros((n, M), device="cuda")
    ids = torch.zeros((n, M, top), dtype=torch.int32, device="cuda")
    tlp = torch.zeros((n, M, top), device="cuda")
    grads = torch.zeros((n, M, V), dtype=torch.bfloat16, device="cuda")
    wait()
    for i in range(n):
        T.quant_fp8(xs[i], 1, out=(codes, scale))
        wait()
        T.matmul_fp8(ws, codes, scale, w, w_scale, out=logits)
        wait()
        T.token_logprobs(lw, logits, tokens, top=top,
                         out=dict(logprob=lp[i], row_stat=stat, top_id=ids[i], top_logprob=tlp[i]))
        wait()
        T.token_logprobs_grad(lw, logits, tokens, stat, g_logprob=weight, out=grads[i])
        wait()
    torch.cuda.synchronize()
    check_no_error(ws)
    check_no_error(lw)
    return lp, ids, tlp, grads


@pytest.mark.parametrize("M,K,V", [(1, 256, 20000), (8, 1024, 6000), (40, 384, 9000), (300, 640, 5000), (2100, 128, 1500)])
def test_chain_without_waits(M, K, V):
    g = torch.Generator(device="cuda").manual_seed(M)
    n = 24 if M < 1000 else 6
    xs = torch.randn((n, M, K), generator=g, device="cuda").to(torch.bfloat16)
    w, w_scale = T.quant_fp8((torch.randn((V, K), generator=g, device="cuda") * (4 / K ** 0.5)).to(torch.bfloat16), 128)
    tokens = torch.randint(0, V, (M,), generator=g, device="cuda", dtype=torch.int32)
    want = _chain(xs, w, w_scale, tokens, torch.cuda.synchronize)
    for _ in range(3):
        got = _chain(xs, w, w_scale, tokens, lambda: None)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_answers_right_behind_the_draft_and_schedule_call():
    """The scheduler ends after the draft kernel it runs beside, so what follows it sees the draft's last rows."""
    wl, s = E.WORKLOAD, E.make()
    n = wl.B * wl.gamma
    lw = T.token_logprobs_workspace(n, wl.V, 3)
    out = None

    def step(wait):
        nonlocal out
        d, _ = T.draft_and_schedule(s["ws"], s["U"], s["W1"], s["W2"], s["h"], s["w"], s["anchor"], s["temp"], s["req_id"],
                                    s["seed"], s["sts"], s["sps"], wl.sched, out=out)
        wait()
        out = d
        r = T.token_logprobs(lw, d["pd_rows"].view(n, wl.V), d["tokens"].reshape(n), top=3)
        torch.cuda.synchronize()
        return {k: v.clone() for k, v in r.items()}

    want = step(torch.cuda.synchronize)
    for _ in range(20):
        out["pd_rows"].zero_()
        got = step(lambda: None)
        for k in want:
            assert torch.equal(got[k], want[k]), k
    check_no_error(s["ws"])
