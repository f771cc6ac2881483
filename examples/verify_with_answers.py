"""One verify step from hidden rows to answers, and one learning step on the same rows.

    python examples/verify_with_answers.py

A served model's vocabulary matrix is laid out once as e4m3 codes with a scale for each 128 x 128
block.  Every step then runs, on one stream and without a host round trip:

    draft_sample -> schedule          the draft block and the rows to verify (a count on the GPU)
    pack_rows                         the target's last hidden rows of those places
    quant_fp8 -> matmul_fp8           their logits (only the counted rows are computed)
    verify                            the emitted tokens
    token_logprobs                    of each emitted token: log probability, rank, entropy, alternatives

and for learning from the answers (here a vocabulary bias raised along the emitted tokens):

    token_logprobs_grad               the gradient of the loss by the logits
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import synth  # noqa: E402
from draft_sampling_lossless_markov_gb300 import capi  # noqa: E402
from draft_sampling_lossless_markov_gb300 import torch_api as T  # noqa: E402

WORKLOAD = synth.Workload("verify_with_answers", 48, 3, 8200, 512, 128, "bf16", "mixed", synth.SCHED_GREEDY, "exp2048",
                          seed=3)


def make(wl=WORKLOAD, device="cuda") -> dict:
    """Synthetic stand-ins for what the model provides, and what a server keeps."""
    s = synth.make_inputs(wl, device, with_target=False)
    g = torch.Generator(device=device).manual_seed(17)
    # the target's last hidden rows of every place (row j of a request predicts place j)
    s["hidden"] = torch.randn((wl.B, wl.gamma + 1, wl.H), generator=g, device=device).to(torch.bfloat16)
    head = (torch.randn((wl.V, wl.H), generator=g, device=device) * (3.0 / wl.H ** 0.5)).to(torch.bfloat16)
    s["head"], s["head_scale"] = T.quant_fp8(head, 128)
    rows = wl.B * (wl.gamma + 1)
    s["ws"] = T.Workspace.create(T.dims(wl.B, wl.gamma, wl.V, wl.r, wl.H, torch.bfloat16), device=device)
    s["ws_mm"] = T.matmul_fp8_workspace(rows, wl.V, wl.H, device=device)
    s["ws_lp"] = T.token_logprobs_workspace(rows, wl.V, 5, device=device)
    s["packed"] = torch.zeros((rows, wl.H), dtype=torch.bfloat16, device=device)
    s["logits"] = torch.zeros((rows, wl.V), dtype=torch.bfloat16, device=device)
    return s


def serve(s: dict, wl=WORKLOAD) -> dict:
    d, sch = T.draft_and_schedule(s["ws"], s["U"], s["W1"], s["W2"], s["h"], s["w"], s["anchor"], s["temp"], s["req_id"],
                                  s["seed"], s["sts"], s["sps"], wl.sched)
    T.pack_rows(s["hidden"], sch["mark_req"], sch["mark_pos"], sch["n_verify"], s["packed"], s["ws"])
    x, x_scale = T.quant_fp8(s["packed"])
    T.matmul_fp8(s["ws_mm"], x, x_scale, s["head"], s["head_scale"], out=s["logits"], n_rows=sch["n_verify"])
    v = T.verify(s["ws"], s["logits"], sch["offsets"], sch["ell"], d["tokens"], d["pd_rows"], d["pd_tok"], s["temp"],
                 s["req_id"], s["seed"])
    a = T.token_logprobs(s["ws_lp"], s["logits"], v["out_tok"], temp=s["temp"], top=5, mark_req=sch["mark_req"],
                         mark_pos=sch["mark_pos"], n_rows=sch["n_verify"])
    return dict(draft=d, schedule=sch, verify=v, answers=a)


def learn(s: dict, r: dict, bias: torch.Tensor, rate: float, wl=WORKLOAD) -> torch.Tensor:
    """One step of raising the mean log probability of the emitted tokens (with a small entropy bonus) by a
    vocabulary bias.  Returns the mean before the step."""
    n = int(r["schedule"]["n_verify"][0])
    rows = (s["logits"][:n].float() + bias).to(torch.bfloat16)
    req, pos = r["schedule"]["mark_req"][:n].contiguous(), r["schedule"]["mark_pos"][:n].contiguous()
    kw = dict(temp=s["temp"], mark_req=req, mark_pos=pos)
    f = T.token_logprobs(s["ws_lp"], rows, r["verify"]["out_tok"], **kw)
    given = int(r["verify"]["n_out"].sum())
    weight = torch.full((n,), 1.0 / given, device=rows.device)
    grad = T.token_logprobs_grad(s["ws_lp"], rows, r["verify"]["out_tok"], f["row_stat"], entropy=f["entropy"],
                                 g_logprob=weight, g_entropy=0.01 * weight, out=rows, **kw)
    bias += rate * grad.float().sum(0)
    return f["logprob"].sum() / given


def main() -> None:
    s = make()
    r = serve(s)
    torch.cuda.synchronize()
    for ws in (s["ws"], s["ws_mm"], s["ws_lp"]):
        code, detail = ws.read_error()
        assert code == 0, (capi.dspark_status_string(code), detail)
    v, a, off = r["verify"], r["answers"], r["schedule"]["offsets"].tolist()
    for q in range(4):
        for j in range(int(v["n_out"][q])):
            i = off[q] + j
            top = " ".join(f"{t}:{p:.2f}" for t, p in zip(a["top_id"][i].tolist(), a["top_logprob"][i].tolist()))
            print(f"request {q} place {j}: token {int(v['out_tok'][q, j])} log p {float(a['logprob'][i]):.3f} "
                  f"rank {int(a['rank'][i])} entropy {float(a['entropy'][i]):.2f} | {top}")
    bias = torch.zeros(WORKLOAD.V, device="cuda")
    means = [float(learn(s, r, bias, 20.0)) for _ in range(5)]
    print("mean log probability of the emitted tokens while the bias learns:", " ".join(f"{m:.3f}" for m in means))


if __name__ == "__main__":
    main()
