"""Workloads of the operators between a served model's last hidden rows and its answers.

Four operators, in the order a verify step or a training step of a vocabulary head uses them:

* ``quant``: rows (or 128 x 128 weight blocks) to 8-bit e4m3 codes, one fp32 scale for each block of 128;
* ``matmul``: the product of two such 8-bit matrices, out[m, n] = sum_b a_scale[m, b] w_scale[n // 128, b]
  sum_{k in block b} a[m, k] w[n, k];
* ``logprobs``: per row of logits the log probability and the rank of a given token, the entropy and the
  top alternatives, at a row's temperature and under a vocabulary mask;
* ``grad``: the gradient of the log probability, the entropy and the top alternatives by the logits.

``run`` with ``own`` false computes them with elementary torch operations in 32 bits; with ``own`` true it
makes the library's calls.  Sizes come from the workloads of synth.py (vocabularies 151936 and 129280,
hidden sizes 2560, 4096 and 7168, 256 requests x 8 verify rows) or are generic.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_MIN = 2.0 ** -100  # a block's largest magnitude counts as at least this
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


def _ceil(a, b):
    return -(-a // b)


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # the activations of a full verify step (256 requests x 8 rows) before the vocabulary projection
        {"name": "quant_step_rows", "op": "quant", "M": 2048, "K": 4096, "dtype": "bf16", "block_rows": 1},
        # a vocabulary matrix laid out once when a model is loaded or after a training step
        {"name": "quant_head_weight", "op": "quant", "M": 151936, "K": 2560, "dtype": "f32", "block_rows": 128},
        # one token of one request through the vocabulary projection: a read of the weights
        {"name": "matmul_one_token_head", "op": "matmul", "M": 1, "K": 2560, "N": 151936, "out": "bf16"},
        # a few rows through a square layer: latency
        {"name": "matmul_few_rows_layer", "op": "matmul", "M": 8, "K": 2560, "N": 2560, "out": "bf16"},
        # 64 requests of one token each on the other vocabulary, logits in full precision
        {"name": "matmul_64_rows_head", "op": "matmul", "M": 64, "K": 7168, "N": 129280, "out": "f32"},
        # the full verify step's logits
        {"name": "matmul_step_head", "op": "matmul", "M": 2048, "K": 4096, "N": 151936, "out": "bf16"},
        # ragged in every direction: no size a multiple of a tile, the last scale block almost empty
        {"name": "matmul_ragged", "op": "matmul", "M": 333, "K": 2050, "N": 10007, "out": "f32"},
        # one emitted token with 20 alternatives: latency
        {"name": "logprobs_one_token", "op": "logprobs", "N": 1, "V": 151936, "dtype": "bf16", "top": 20, "mask": False},
        # every row of a full verify step with 8 alternatives, mixed temperatures
        {"name": "logprobs_step", "op": "logprobs", "N": 2048, "V": 151936, "dtype": "bf16", "top": 8, "mask": False},
        # constrained decoding: odd vocabulary, a mask a row, some rows with nothing left
        {"name": "logprobs_masked_odd", "op": "logprobs", "N": 301, "V": 100003, "dtype": "f32", "top": 5, "mask": True},
        # policy-gradient step over the same rows: log probability and entropy bonus
        {"name": "grad_step", "op": "grad", "N": 2048, "V": 151936, "dtype": "bf16", "top": 0, "mask": False},
        # distillation on the alternatives under a mask, odd vocabulary
        {"name": "grad_masked_odd", "op": "grad", "N": 301, "V": 100003, "dtype": "f32", "top": 5, "mask": True},
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, even over the logarithm; odd sizes and multiples of 8 are both common."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        n = max(lo, n // 8 * 8)
    n = min(hi, max(lo, n))
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["quant", "matmul", "matmul", "logprobs", "logprobs", "grad"])
    if op == "quant":
        while True:
            c = {"op": op, "M": _spread(rng, 1, 152000), "K": _spread(rng, 64, 8192), "dtype": rng.choice(["bf16", "f32"]),
                 "block_rows": rng.choice([1, 128])}
            if c["M"] * c["K"] <= 151936 * 2560:
                return c
    if op == "matmul":
        while True:
            c = {"op": op, "M": _spread(rng, 1, 4096), "K": _spread(rng, 64, 8192), "N": _spread(rng, 128, 152000),
                 "out": rng.choice(["bf16", "f32"])}
            if c["M"] * c["K"] * c["N"] <= 2048 * 4096 * 151936 and c["M"] * c["N"] * BYTES[c["out"]] <= 2048 * 151936 * 2:
                return c
    while True:
        c = {"op": op, "N": _spread(rng, 1, 4096), "V": _spread(rng, 1000, 200000), "dtype": rng.choice(["bf16", "f32"]),
             "top": rng.choice([0, 1, 5, 20, 32]), "mask": rng.random() < 0.4}
        if c["N"] * c["V"] * BYTES[c["dtype"]] <= 2048 * 151936 * 2:
            return c


# --------------------------------------------------------------------------- inputs
def _gen(seed, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 16 + k)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _codes_buffer(rows, cols):
    """Rows of 8-bit codes; the stride between rows is a multiple of 16 bytes."""
    return torch.zeros((rows, _ceil(cols, 16) * 16), dtype=torch.float8_e4m3fn, device="cuda")[:, :cols]


def _make_codes(g, rows, cols, block_rows, spread):
    """Codes and scales of a random matrix, as a quantised checkpoint or the step before holds them."""
    x = _randn(g, rows, cols)
    if spread:  # some hidden channels are much larger than the others
        x.mul_(torch.exp(0.7 * _randn(g, cols)))
    else:
        x.mul_(0.02)
    q, s = _quant_plain(x, block_rows)
    codes = _codes_buffer(rows, cols)
    codes.copy_(q)
    return codes, s


def _logit_inputs(case, seed):
    N, V = case["N"], case["V"]
    g = _gen(seed, 3)
    z = _randn(g, N, V)
    z.mul_(3.0).sub_(1.1 * torch.log(torch.arange(V, device="cuda", dtype=torch.float32) + 1.0))
    s = {"logits": z.to(DTYPES[case["dtype"]]).contiguous()}
    u = torch.rand((N,), generator=g, device="cuda")
    tok = (u.pow(3) * V).long().clamp_(max=V - 1).to(torch.int32)
    gone = torch.rand((N,), generator=g, device="cuda") < 0.05  # rows past a rejection have no token
    s["tokens"] = torch.where(gone, torch.full_like(tok, -1), tok)
    pick = torch.randint(0, 3, (N,), generator=g, device="cuda")
    s["temp"] = torch.tensor([0.0, 0.7, 1.0], device="cuda")[pick]  # 0: greedy, answered at temperature 1
    if case["mask"]:
        words = torch.randint(-2 ** 31, 2 ** 31, (N, _ceil(V, 32)), generator=g, device="cuda", dtype=torch.int64)
        words = words.to(torch.int32)
        words[torch.rand((N,), generator=g, device="cuda") < 1 / 16] = 0
        s["mask"] = words
    else:
        s["mask"] = None
    return s, g


def prepare(case, seed):
    op = case["op"]
    s = {"op": op, "case": dict(case)}
    if op == "quant":
        g = _gen(seed, 1)
        x = _randn(g, case["M"], case["K"])
        x.mul_(torch.exp(0.7 * _randn(g, case["K"])))
        s["x"] = x.to(DTYPES[case["dtype"]])
        s["out"] = (_codes_buffer(case["M"], case["K"]),
                    torch.empty((_ceil(case["M"], case["block_rows"]), _ceil(case["K"], BLOCK)), device="cuda"))
        return s
    if op == "matmul":
        g = _gen(seed, 2)
        s["a"], s["a_scale"] = _make_codes(g, case["M"], case["K"], 1, True)
        s["w"], s["w_scale"] = _make_codes(g, case["N"], case["K"], 128, False)
        s["out"] = torch.empty((case["M"], case["N"]), dtype=DTYPES[case["out"]], device="cuda")
        if own:
            from draft_sampling_lossless_markov_gb300 import torch_api as T
            s["ws"] = T.matmul_fp8_workspace(case["M"], case["N"], case["K"])
        return s
    t, g = _logit_inputs(case, seed)
    s.update(t)
    N, V, top = case["N"], case["V"], case["top"]
    if op == "grad":  # what the forward pass kept, and the loss's gradients by its outputs
        f = _logprobs_plain(s["logits"], s["tokens"], s["temp"], top, s["mask"])
        s["row_stat"], s["entropy"], s["top_id"] = f["row_stat"], f["entropy"], f["top_id"]
        s["g_logprob"] = _randn(g, N) / N
        s["g_entropy"] = 0.01 * _randn(g, N) / N
        s["g_top"] = _randn(g, N, top) / N if top else None
        s["out"] = torch.empty_like(s["logits"])
    else:
        f32 = dict(dtype=torch.float32, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        s["out"] = dict(logprob=torch.empty(N, **f32), entropy=torch.empty(N, **f32), rank=torch.empty(N, **i32),
                        row_stat=torch.empty((N, 2), **f32), top_id=torch.empty((N, top), **i32),
                        top_logprob=torch.empty((N, top), **f32))
    if own:
        from draft_sampling_lossless_markov_gb300 import torch_api as T
        s["ws"] = T.token_logprobs_workspace(N, V, top)
    return s


# --------------------------------------------------------------------------- the plain forms, in 32 bits
def _quant_plain(x, block_rows):
    rows, cols = x.shape
    kb, rb = _ceil(cols, BLOCK), _ceil(rows, block_rows)
    v = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - cols, 0, rb * block_rows - rows))
    v = v.view(rb, block_rows, kb, BLOCK)
    amax = v.abs().amax(dim=(1, 3)).clamp(min=AMAX_MIN)
    inv = E4M3_MAX / amax
    q = (v * inv[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(rb * block_rows, kb * BLOCK)[:rows, :cols], amax / E4M3_MAX


def _dequant(q, scale, block_rows):
    rows, cols = q.shape
    s = scale.repeat_interleave(block_rows, 0)[:rows] if block_rows > 1 else scale
    return q.float() * s.repeat_interleave(BLOCK, 1)[:, :cols]


def _allowed(logits, mask):
    ok = logits > -math.inf
    if mask is not None:
        N, V = logits.shape
        bits = torch.arange(32, device=logits.device, dtype=torch.int32)
        ok = ok & ((mask[:, :, None] >> bits) & 1).bool().view(N, -1)[:, :V]
    return ok


def _logprobs_plain(logits, tokens, temp, top, mask):
    N, V = logits.shape
    z = logits.float()
    ok = _allowed(z, mask)
    t = torch.where((temp > 0) & torch.isfinite(temp), temp, torch.ones_like(temp))[:, None]
    z = z.masked_fill(~ok, -math.inf)
    m = z.amax(1, keepdim=True)
    some = m > -math.inf
    d = (z - torch.where(some, m, torch.zeros_like(m))) / t
    e = torch.exp(d)
    S = e.sum(1, keepdim=True)
    logS = torch.log(S)
    H = torch.where(some, logS - torch.where(ok, e * d, torch.zeros_like(e)).sum(1, keepdim=True) / S,
                    torch.zeros_like(S))[:, 0]
    given = tokens >= 0
    at = tokens.clamp(min=0).long()[:, None]
    lp = torch.where(some, d.gather(1, at) - logS, torch.full_like(S, -math.inf))[:, 0]
    zt = z.gather(1, at)
    ids = torch.arange(V, device=z.device)
    ahead = ((z > zt) | ((z == zt) & (ids < at))).sum(1)
    rank = torch.where(given & (zt[:, 0] > -math.inf), ahead, torch.full_like(ahead, -1)).to(torch.int32)
    out = {"logprob": torch.where(given, lp, torch.zeros_like(lp)), "entropy": H, "rank": rank,
           "row_stat": torch.cat([m, S], 1)}
    # one whole number orders by (logit descending, id ascending); + 0.0 makes -0 equal 0
    b = (z + 0.0).view(torch.int32)
    key = torch.where(b < 0, b ^ 0x7FFFFFFF, b).long() * 2 ** 32 + (0x7FFFFFFF - ids)
    key = key.masked_fill(~ok, -2 ** 63)
    best, _ = torch.topk(key, min(top, V), dim=1)
    best = torch.nn.functional.pad(best, (0, top - best.shape[1]), value=-2 ** 63)
    found = best > -2 ** 63
    tid = torch.where(found, 0x7FFFFFFF - (best & 0xFFFFFFFF), torch.full_like(best, -1))
    out["top_id"] = tid.to(torch.int32)
    out["top_logprob"] = torch.where(found, d.gather(1, tid.clamp(min=0)) - logS,
                                     torch.full_like(best, -math.inf, dtype=torch.float32))
    return out


def _grad_plain(s):
    z = s["logits"].float()
    ok = _allowed(z, s["mask"])
    temp = s["temp"]
    t = torch.where((temp > 0) & torch.isfinite(temp), temp, torch.ones_like(temp))[:, None]
    m, S = s["row_stat"][:, :1], s["row_stat"][:, 1:]
    some = m > -math.inf
    live = ok & some
    logp = (z - torch.where(some, m, torch.zeros_like(m))) / t - torch.log(S)
    logp = torch.where(live, logp, torch.zeros_like(logp))
    p = torch.where(live, torch.exp(logp), torch.zeros_like(logp))
    at = s["tokens"].clamp(min=0).long()[:, None]
    has = (s["tokens"] >= 0)[:, None] & ok.gather(1, at)
    g = torch.where(has, s["g_logprob"][:, None], torch.zeros_like(m))
    total, pick = g, torch.zeros_like(p).scatter_add_(1, at, g)
    if s["g_top"] is not None:
        gt = torch.where(s["top_id"] >= 0, s["g_top"], torch.zeros_like(s["g_top"]))
        total = total + gt.sum(1, keepdim=True)
        pick.scatter_add_(1, s["top_id"].clamp(min=0).long(), gt)
    dz = (pick - p * (total + s["g_entropy"][:, None] * (logp + s["entropy"][:, None]))) / t
    return torch.where(live, dz, torch.zeros_like(dz)).to(s["logits"].dtype)


def run(s):
    op, c = s["op"], s["case"]
    if own:
        from draft_sampling_lossless_markov_gb300 import torch_api as T
        if op == "quant":
            return T.quant_fp8(s["x"], c["block_rows"], out=s["out"])
        if op == "matmul":
            return T.matmul_fp8(s["ws"], s["a"], s["a_scale"], s["w"], s["w_scale"], out=s["out"])
        if op == "logprobs":
            return T.token_logprobs(s["ws"], s["logits"], s["tokens"], temp=s["temp"], top=c["top"], mask=s["mask"],
                                    out=s["out"])
        return T.token_logprobs_grad(s["ws"], s["logits"], s["tokens"], s["row_stat"], entropy=s["entropy"],
                                     top_id=s["top_id"], g_logprob=s["g_logprob"], g_entropy=s["g_entropy"],
                                     g_top=s["g_top"], temp=s["temp"], mask=s["mask"], out=s["out"])
    if op == "quant":
        return _quant_plain(s["x"], c["block_rows"])
    if op == "matmul":
        return torch.matmul(_dequant(s["a"], s["a_scale"], 1), _dequant(s["w"], s["w_scale"], 128).t()).to(DTYPES[c["out"]])
    if op == "logprobs":
        return _logprobs_plain(s["logits"], s["tokens"], s["temp"], c["top"], s["mask"])
    return _grad_plain(s)


# --------------------------------------------------------------------------- the definition, in 64 bits
def _e4m3(v):
    """The e4m3 value nearest to v (ties to even, at most 448), for float64 v."""
    a = v.abs()
    _, e = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), torch.clamp(e - 1, min=-6) - 3)
    return torch.copysign(torch.clamp(torch.round(a / step) * step, max=E4M3_MAX), v)


def _exact_quant(x, block_rows):
    M, K = x.shape
    codes = torch.empty((M, K), dtype=torch.float64, device=x.device)
    scales = torch.empty((_ceil(M, block_rows), _ceil(K, BLOCK)), dtype=torch.float64, device=x.device)
    for b in range(scales.shape[1]):
        part = x[:, b * BLOCK:(b + 1) * BLOCK].double()
        rowmax = part.abs().amax(1)
        rowmax = torch.cat([rowmax, rowmax.new_zeros(scales.shape[0] * block_rows - M)])
        amax = torch.maximum(rowmax.view(-1, block_rows).amax(1), rowmax.new_tensor(AMAX_MIN))
        scales[:, b] = amax / E4M3_MAX
        codes[:, b * BLOCK:(b + 1) * BLOCK] = _e4m3(part * (E4M3_MAX / amax).repeat_interleave(block_rows)[:M, None])
    return codes, scales


def _exact_matmul(s):
    a, w = s["a"], s["w"]
    (M, K), N = a.shape, w.shape[0]
    which = torch.arange(K, device=a.device) // BLOCK
    ad = a.to(torch.float64) * s["a_scale"].double()[:, which]
    out = torch.empty((M, N), dtype=torch.float64, device=a.device)
    for n0 in range(0, N, 8192):
        rows = torch.arange(n0, min(N, n0 + 8192), device=a.device)
        wd = w[n0:n0 + 8192].to(torch.float64) * s["w_scale"].double()[rows // BLOCK][:, which]
        out[:, n0:n0 + 8192] = ad @ wd.T
    return out


def _bits(mask, V):
    """Boolean [rows, V] of the mask's little-endian bits."""
    by = mask.contiguous().view(torch.uint8)
    sel = torch.tensor([1, 2, 4, 8, 16, 32, 64, 128], dtype=torch.uint8, device=mask.device)
    return ((by[:, :, None] & sel) != 0).flatten(1)[:, :V]


def _exact_rows(s, lo, hi):
    """Shifted log weights, normaliser and candidates of rows lo..hi, in 64 bits."""
    z = s["logits"][lo:hi].double()
    if s["mask"] is not None:
        z = torch.where(_bits(s["mask"][lo:hi], z.shape[1]), z, z.new_tensor(-math.inf))
    T = s["temp"][lo:hi].double()
    T = torch.where(T > 0, T, torch.ones_like(T))[:, None]
    logp = torch.log_softmax(z / T, 1)  # NaN where nothing is left
    return z, T, logp, torch.isneginf(z).all(1)


def _exact_logprobs(s, case):
    N, V = s["logits"].shape
    top = case["top"]
    parts = []
    for lo in range(0, N, 64):
        z, T, logp, empty = _exact_rows(s, lo, lo + 64)
        n = z.shape[0]
        tok = s["tokens"][lo:lo + 64].long()
        r = torch.arange(n, device=z.device)
        safe = torch.where(empty[:, None], torch.full_like(logp, -math.inf), logp)
        lp = torch.where(tok >= 0, safe[r, tok.clamp(min=0)], torch.zeros(n, dtype=torch.float64, device=z.device))
        p = torch.exp(safe)
        H = -torch.where(p > 0, p * safe, torch.zeros_like(p)).sum(1)
        mx = z.max(1).values
        S = torch.where(empty, torch.zeros_like(mx), torch.exp((z - torch.where(empty, 0 * H, mx)[:, None]) / T).sum(1))
        zt = z[r, tok.clamp(min=0)][:, None]
        below = torch.arange(V, device=z.device)[None] < tok[:, None]
        rank = (z > zt).sum(1) + ((z == zt) & below).sum(1)
        rank = torch.where((tok >= 0) & ~torch.isneginf(zt[:, 0]), rank, torch.full_like(rank, -1))
        tid = torch.full((n, top), -1, dtype=torch.int64, device=z.device)
        tlp = torch.full((n, top), -math.inf, dtype=torch.float64, device=z.device)
        if top:
            order = torch.sort(z, dim=1, descending=True, stable=True)
            k = min(top, V)
            good = ~torch.isneginf(order.values[:, :k])
            tid[:, :k] = torch.where(good, order.indices[:, :k], tid[:, :k])
            tlp[:, :k] = torch.where(good, safe.gather(1, order.indices[:, :k]), tlp[:, :k])
        parts.append((lp, H, rank.to(torch.int32), torch.stack([mx, S], 1), tid.to(torch.int32), tlp))
    names = ("logprob", "entropy", "rank", "row_stat", "top_id", "top_logprob")
    return {n: torch.cat(x) for n, x in zip(names, zip(*parts))}


def _exact_grad(s):
    N, V = s["logits"].shape
    out = torch.empty((N, V), dtype=torch.float64, device="cuda")
    for lo in range(0, N, 64):
        z, T, logp, empty = _exact_rows(s, lo, lo + 64)
        n = z.shape[0]
        r = torch.arange(n, device=z.device)
        safe = torch.where(torch.isneginf(z), torch.zeros_like(logp), logp)  # 0 log 0 = 0
        p = torch.where(torch.isneginf(z), torch.zeros_like(logp), torch.exp(logp))
        H = -(p * safe).sum(1, keepdim=True)
        # rows of the Jacobian of each output, weighted by the gradient by it
        d = -s["g_entropy"][lo:lo + 64].double()[:, None] * p * (safe + H)
        picks = [(s["tokens"][lo:lo + 64].long(), s["g_logprob"][lo:lo + 64].double())]
        if s["g_top"] is not None:
            picks += [(s["top_id"][lo:lo + 64, k].long(), s["g_top"][lo:lo + 64, k].double()) for k in range(s["g_top"].shape[1])]
        for at, g in picks:
            at0 = at.clamp(min=0)
            g = torch.where((at >= 0) & ~torch.isneginf(z[r, at0]), g, torch.zeros_like(g))
            d -= g[:, None] * p
            d[r, at0] += g
        d = torch.where(torch.isneginf(z) | empty[:, None], torch.zeros_like(d), d / T)
        out[lo:lo + 64] = d
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        return _exact_quant(s["x"], case["block_rows"])
    if case["op"] == "matmul":
        return _exact_matmul(s)
    if case["op"] == "logprobs":
        return _exact_logprobs(s, case)
    return _exact_grad(s)


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "quant":
        n = case["M"] * case["K"]
        scales = _ceil(case["M"], case["block_rows"]) * _ceil(case["K"], BLOCK) * 4
        return {"bytes": n * (BYTES[case["dtype"]] + 1) + scales, "flops": 3 * n}
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        kb = _ceil(K, BLOCK)
        return {"bytes": M * K + N * K + 4 * kb * (M + _ceil(N, 128)) + M * N * BYTES[case["out"]], "flops": 2 * M * N * K}
    N, V, top = case["N"], case["V"], case["top"]
    mask = N * _ceil(V, 32) * 4 if case["mask"] else 0
    if op == "logprobs":
        return {"bytes": N * V * BYTES[case["dtype"]] + mask + N * (8 + 20 + 8 * top), "flops": 6 * N * V}
    return {"bytes": 2 * N * V * BYTES[case["dtype"]] + mask + N * (28 + 8 * top), "flops": 6 * N * V}
