"""Decode steps of a small target with one attention layer over a paged e4m3 cache.

    python examples/decode_with_cache.py

The weights and the draft's inputs are random stand-ins; the calls are those of a served step, on one
stream and without a host round trip:

    draft_sample -> schedule          the draft block and the rows to verify (a count on the GPU)
    quant_fp8 -> matmul_fp8           queries, keys and values of the rows' tokens
    cache_write                       the drafted rows' keys and values, behind each request's context
    tree_attention                    every row over the context and the drafted rows up to itself
    quant_fp8 -> matmul_fp8           the layer's output, and the logits
    verify                            the emitted tokens; the accepted rows stay in the cache

A chain's accepted rows lie where they belong.  Of a tree's, `keep_path` moves those on the accepted path
behind the context (cache_move).
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import synth  # noqa: E402
from draft_sampling_lossless_markov_gb300 import capi  # noqa: E402
from draft_sampling_lossless_markov_gb300 import torch_api as T  # noqa: E402

WORKLOAD = synth.Workload("decode_with_cache", 24, 3, 8200, 512, 128, "bf16", "mixed", synth.SCHED_GREEDY, "exp2048", seed=4)
HQ, HKV, D, PAGE = 8, 2, 128, 16
BF16, I32 = torch.bfloat16, torch.int32


def make(wl=WORKLOAD, prompt=40, room=128, device="cuda") -> dict:
    """What the model provides, and what a server keeps: weights as codes, the cache, workspaces, buffers."""
    s = synth.make_inputs(wl, device, with_target=False)
    g = torch.Generator(device=device).manual_seed(23)
    rand = lambda *shape: torch.randn(shape, generator=g, device=device)  # noqa: E731
    rows = wl.B * (wl.gamma + 1)
    s["embedding"] = rand(wl.V, wl.H).to(BF16)
    for name, n, k in (("qkv", (HQ + 2 * HKV) * D, wl.H), ("o", wl.H, HQ * D), ("head", wl.V, wl.H)):
        s["w_" + name], s["s_" + name] = T.quant_fp8((rand(n, k) * k ** -0.5).to(BF16), 128)
        s["ws_" + name] = T.matmul_fp8_workspace(max(rows, wl.B * prompt), n, k, device=device)
    s["ws"] = T.Workspace.create(T.dims(wl.B, wl.gamma, wl.V, wl.r, wl.H, BF16), device=device)
    s["ws_attn"] = T.tree_attention_workspace(wl.B, wl.gamma + 1, HQ, HKV, D, device=device)
    pages = -(-(prompt + room) // PAGE)
    table = torch.randperm(wl.B * pages, generator=g, device=device).to(I32).view(wl.B, pages)
    s["cache"] = T.KvCache.create(wl.B * pages, PAGE, HKV, D, table)
    s["base"] = torch.full((wl.B,), prompt, dtype=I32, device=device)
    s["attended"] = torch.zeros((rows, HQ, D), dtype=BF16, device=device)
    # the prompts' keys and values: their rows' marks count from position 0
    tokens = torch.randint(0, wl.V, (wl.B * prompt,), generator=g, device=device)
    _, k, v = project(s, s["embedding"][tokens])
    i = torch.arange(wl.B * prompt, device=device, dtype=I32)
    T.cache_write(s["cache"], k, v, i // prompt, i % prompt, ws=s["ws"])
    return s


def product(s: dict, name: str, x: torch.Tensor, n_rows=None) -> torch.Tensor:
    codes, scale = T.quant_fp8(x)
    out = torch.empty((x.shape[0], s["w_" + name].shape[0]), dtype=BF16, device=x.device)
    return T.matmul_fp8(s["ws_" + name], codes, scale, s["w_" + name], s["s_" + name], out=out, n_rows=n_rows)


def project(s: dict, x: torch.Tensor, n_rows=None) -> tuple:
    """(q, k, v) of rows x, as views of one product."""
    y = product(s, "qkv", x, n_rows)
    return tuple(y[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, HQ), (HQ, HQ + HKV), (HQ + HKV, HQ + 2 * HKV)))


def step(s: dict, wl=WORKLOAD) -> dict:
    d, sch = T.draft_and_schedule(s["ws"], s["U"], s["W1"], s["W2"], s["h"], s["w"], s["anchor"], s["temp"], s["req_id"],
                                  s["seed"], s["sts"], s["sps"], wl.sched)
    n = sch["n_verify"]
    x = s["embedding"][sch["flat_tok"].clamp(0, wl.V - 1).long()]
    q, k, v = project(s, x, n)
    T.cache_write(s["cache"], k, v, sch["mark_req"], sch["mark_pos"], base=s["base"], n_rows=n, ws=s["ws"])
    T.tree_attention(s["ws_attn"], s["cache"], q, sch["offsets"], s["base"], wl.gamma + 1, out=s["attended"])
    x = x + product(s, "o", s["attended"].flatten(1), n)
    logits = product(s, "head", x, n)
    r = T.verify(s["ws"], logits, sch["offsets"], sch["ell"], d["tokens"], d["pd_rows"], d["pd_tok"], s["temp"], s["req_id"],
                 s["seed"])
    # the next step begins at the last emitted token, whose row the cache does not hold yet
    before = s["base"].clone()
    s["base"] += r["n_out"]
    s["anchor"] = r["out_tok"].gather(1, (r["n_out"] - 1).long()[:, None])[:, 0].to(s["anchor"].dtype)
    s["seed"] += 1
    return dict(schedule=sch, verify=r, q=q, base=before)


def keep_path(s: dict, base: torch.Tensor, nodes: torch.Tensor, count: torch.Tensor) -> None:
    """Of drafted trees written behind base: the rows of nodes[r, :count[r]] become the context's next."""
    T.cache_move(s["cache"], base, nodes, count, ws=s["ws"])


def main() -> None:
    s = make()
    emitted = torch.zeros_like(s["base"])
    for _ in range(5):
        emitted += step(s)["verify"]["n_out"]
    torch.cuda.synchronize()
    for name, ws in s.items():
        if isinstance(ws, T.Workspace):
            code, detail = ws.read_error()
            assert code == 0, (name, capi.dspark_status_string(code), detail)
    print("tokens emitted in 5 steps:", emitted.tolist())
    print("context lengths:", s["base"].tolist())


if __name__ == "__main__":
    main()
