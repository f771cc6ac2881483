"""The serving and learning example end to end: the answers agree with the fp64 oracle on the logits the
projection made, and those with the oracle's product."""
import numpy as np
import pytest
import torch

from examples import verify_with_answers as E
from gpu_common import check_no_error, require_gpu
from oracle import vocab as O

pytestmark = pytest.mark.gpu


def test_verify_step_with_answers():
    require_gpu()
    s = E.make()
    r = E.serve(s)
    torch.cuda.synchronize()
    for ws in (s["ws"], s["ws_mm"], s["ws_lp"]):
        check_no_error(ws)
    wl, sch, a = E.WORKLOAD, r["schedule"], r["answers"]
    n = int(sch["n_verify"][0])
    assert wl.B <= n <= wl.B * (wl.gamma + 1)
    f64 = lambda t: t.detach().to("cpu", torch.float64).numpy()  # noqa: E731
    # the logits of a few packed rows: e4m3 rounding (2^-4 of each factor) is part of the definition, so the
    # oracle multiplies the same codes; bf16 rounds the result (2^-8)
    rows = np.unique(np.linspace(0, n - 1, 7).astype(int))
    scaled, scale = O.quant(f64(s["packed"][rows]), 1)
    head = O.dequant(s["head"].contiguous().view(torch.uint8).cpu().numpy(), f64(s["head_scale"]), 128)
    x = O.e4m3_round(scaled) * scale[:, np.arange(wl.H) // 128]
    want = x @ head.T
    got = f64(s["logits"][rows])
    # a code may fall on the other side of a tie: 2^-3 of one factor, of at most a few of 512 terms
    slack = 2.0 ** -8 * np.abs(want) + 3 * 2.0 ** -3 * np.abs(x).max(1)[:, None] * np.abs(head).max(1)[None] + 1e-30
    assert (np.abs(got - want) <= slack).all()
    assert np.median(np.abs(got - want) / (np.abs(want) + 1e-6)) < 2.0 ** -8
    # the answers on those logits
    req, pos = sch["mark_req"].cpu().numpy()[:n], sch["mark_pos"].cpu().numpy()[:n]
    tok = r["verify"]["out_tok"].cpu().numpy()[req, pos]
    temp = s["temp"].cpu().numpy()[req]
    ref = O.token_logprobs(f64(s["logits"][:n]), tok, temp, 5)
    np.testing.assert_array_equal(a["rank"].cpu().numpy()[:n], ref["rank"])
    np.testing.assert_array_equal(a["top_id"].cpu().numpy()[:n], ref["top_id"])
    np.testing.assert_allclose(f64(a["logprob"])[:n], ref["logprob"], atol=1e-4)
    np.testing.assert_allclose(f64(a["entropy"])[:n], ref["entropy"], atol=1e-3)
    assert (tok >= 0).sum() == int(r["verify"]["n_out"].sum())


def test_learning_raises_the_emitted_tokens():
    require_gpu()
    s = E.make()
    r = E.serve(s)
    bias = torch.zeros(E.WORKLOAD.V, device="cuda")
    means = [float(E.learn(s, r, bias, 20.0)) for _ in range(6)]
    assert all(b > a for a, b in zip(means, means[1:]))
    # the first step's gradient by the bias is the sum of the rows' gradients
    assert abs(float(bias.sum())) < 1e-2 * float(bias.abs().sum())
