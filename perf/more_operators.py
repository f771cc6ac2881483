"""Workloads of the operators around a served model's key/value cache.

Four operators, in the order a verify step uses them:

* ``write``: keys and values of new rows to a paged cache, as e4m3 codes with one fp32 scale for each row and head, or bf16;
* ``attn``: attention of every request's drafted rows (a chain, or a tree given by one bit mask a row) over its cached
  context and the drafted rows before them, from the cache;
* ``move``: the accepted path of a tree goes to the places behind the context;
* ``read``: cached rows back as bf16 or fp32.

The cache has pages of ``page`` tokens: k and v [pages, kv heads, page, head size], scales [pages, kv heads, page];
position p of request r is slot p % page of page table[r, p // page].  ``run`` with ``own`` false computes the operators
with elementary torch operations in 32 bits; with ``own`` true it makes the library's calls.  Row counts come from the
workloads of synth.py (256 requests x 8 verify rows, 64 x 8, 16 rows a request), the rest is generic.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
AMAX_MIN = 2.0 ** -100  # a row's largest magnitude counts as at least this
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
CODE_BYTES = {"e4m3": 1, "bf16": 2}


def _ceil(a, b):
    return -(-a // b)


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one request: latency
        {"name": "attn_one_token", "op": "attn", "B": 1, "rows": 1, "Hq": 32, "Hkv": 8, "D": 128, "L": 1000, "page": 64,
         "cache": "e4m3", "tree": False},
        # a full verify step: 256 requests x 8 rows, contexts of every length up to 8192
        {"name": "attn_step", "op": "attn", "B": 256, "rows": 8, "Hq": 32, "Hkv": 8, "D": 128, "L": 8192, "page": 64,
         "cache": "e4m3", "tree": False},
        # 16 rows a request over a cache kept in 16 bits
        {"name": "attn_step_bf16", "op": "attn", "B": 64, "rows": 16, "Hq": 32, "Hkv": 8, "D": 128, "L": 4096, "page": 128,
         "cache": "bf16", "tree": False},
        # one request with a long context: the long axis has to be split
        {"name": "attn_long", "op": "attn", "B": 1, "rows": 8, "Hq": 32, "Hkv": 8, "D": 128, "L": 250001, "page": 32,
         "cache": "e4m3", "tree": False},
        # wide trees: 64 drafted nodes x 8 query heads on every cached row
        {"name": "attn_tree", "op": "attn", "B": 16, "rows": 64, "Hq": 64, "Hkv": 8, "D": 128, "L": 6000, "page": 16,
         "cache": "e4m3", "tree": True},
        # ragged in everything: requests without rows, empty contexts, 7 query heads a kv head, the smaller head size
        {"name": "attn_odd", "op": "attn", "B": 37, "rows": 13, "Hq": 14, "Hkv": 2, "D": 64, "L": 1777, "page": 16,
         "cache": "e4m3", "tree": True},
        # the drafted rows of a full verify step
        {"name": "write_step", "op": "write", "B": 256, "rows": 8, "Hkv": 8, "D": 128, "page": 64, "cache": "e4m3",
         "dtype": "bf16"},
        # prompts
        {"name": "write_prompts", "op": "write", "B": 16, "rows": 4096, "Hkv": 8, "D": 128, "page": 64, "cache": "e4m3",
         "dtype": "bf16"},
        # whole contexts back, to hand them on
        {"name": "read_contexts", "op": "read", "B": 16, "rows": 4096, "Hkv": 8, "D": 128, "page": 64, "cache": "e4m3",
         "dtype": "bf16"},
        # some rows of few heads in full precision
        {"name": "read_odd", "op": "read", "B": 37, "rows": 81, "Hkv": 3, "D": 64, "page": 16, "cache": "e4m3", "dtype": "f32"},
        # the accepted paths of a step's trees
        {"name": "move_step", "op": "move", "B": 256, "rows": 8, "Hkv": 8, "D": 128, "page": 64, "cache": "e4m3"},
        # many requests, long paths, 16 bits
        {"name": "move_many", "op": "move", "B": 2000, "rows": 16, "Hkv": 8, "D": 128, "page": 32, "cache": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, even over the logarithm; odd sizes and multiples of 8 are both common."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.3:
        n = max(lo, n // 8 * 8)
    return min(hi, max(lo, n))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "attn", "write", "read", "move"])
    c = {"op": op, "D": rng.choice([64, 128, 128]), "page": rng.choice([16, 32, 64, 128]),
         "cache": rng.choice(["e4m3", "e4m3", "bf16"]), "Hkv": rng.choice([1, 2, 3, 4, 8, 8, 16])}
    if op == "attn":
        limit = [work(x) for x in listed()]
        while True:
            c.update(B=_spread(rng, 1, 256), rows=_spread(rng, 1, 64), L=_spread(rng, 1, 250000), tree=rng.random() < 0.5)
            c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 16])
            w = work(c)
            padded = c["B"] * (c["L"] + c["rows"]) * max(c["Hkv"] * c["D"], c["Hq"] * c["rows"])  # of the plain form's products
            if w["bytes"] <= max(x["bytes"] for x in limit[:6]) and w["flops"] <= max(x["flops"] for x in limit[:6]) and \
                    padded <= 256 * 8192 * 8 * 256:
                return c
    if op != "move":
        c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
    while True:
        c.update(B=_spread(rng, 1, 2000), rows=_spread(rng, 1, 32 if op == "move" else 8192))
        if work(c)["bytes"] <= work(listed()[7])["bytes"]:
            return c


# --------------------------------------------------------------------------- lengths, the same for every seed but for their order
def _contexts(case):
    """Cached tokens of each request before its drafted rows, spread over 0 .. L (one request: L)."""
    B, L = case["B"], case["L"]
    return [L] if B == 1 else [int(L * ((r * 0.6180339887498949 + 0.37) % 1.0)) if r % 19 != 7 else (0, L)[r // 19 % 2] for r in range(B)]


def _row_counts(case):
    """Rows of each request: all of them for chains of a fixed length, 0 .. rows for trees."""
    B, R = case["B"], case["rows"]
    if not case.get("tree") or B == 1:
        return [R] * B
    return [R - int((R + 1) * ((r * 0.7548776662466927) % 1.0)) if r % 3 else R for r in range(B)]


def _path_counts(case):
    return [1 + r % case["rows"] for r in range(case["B"])]


# --------------------------------------------------------------------------- inputs
def _gen(seed, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 16 + k)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _places(counts):
    """(request, place within it) of every row."""
    n = torch.tensor(counts, dtype=torch.int64, device="cuda")
    req = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), n)
    return req, torch.arange(req.numel(), device="cuda") - (torch.cumsum(n, 0) - n)[req]


def _make_cache(g, case, tokens):
    """A pool with room for tokens[r] of every request r, its pages dealt out in random order, filled with normal
    rows; the scales of 8-bit rows differ from row to row."""
    P, H, D = case["page"], case["Hkv"], case["D"]
    per = [_ceil(t, P) for t in tokens]
    total = sum(per) + 3
    s = {"page": P, "n_pages": total}
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(per), max(1, max(per))), -1, dtype=torch.int32, device="cuda")
    req, at = _places(per)
    table[req, at] = order[:req.numel()]
    s["table"] = table
    shape = (total, H, P)
    if case["cache"] == "bf16":
        for name in ("k", "v"):
            s[name] = torch.empty(shape + (D,), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
            s[name + "_scale"] = None
    else:
        for name in ("k", "v"):  # codes of normal rows whose largest is at 448
            x = torch.empty(shape + (D,), dtype=torch.bfloat16, device="cuda").normal_(generator=g).mul_(150.0).clamp_(-448.0, 448.0)
            s[name] = x.to(torch.float8_e4m3fn)
            s[name + "_scale"] = torch.exp(0.3 * torch.randn(shape, generator=g, device="cuda")) / 150.0
    return s


def _random_tree(g, req, place):
    """One mask of 64 bits a row: itself and its ancestors; the parent of node j is one of the nodes before it."""
    n = place.numel()
    B = int(req.max()) + 1 if n else 0
    R = int(place.max()) + 1 if n else 0
    u = torch.rand((B, R), generator=g, device="cuda")
    bits = torch.zeros((B, R), dtype=torch.int64, device="cuda")
    rows = torch.arange(B, device="cuda")
    for j in range(R):  # nodes in order, every tree at once
        bits[:, j] = 1 << j if j < 63 else -2 ** 63
        if j:
            bits[:, j] |= bits[rows, (u[:, j] * j).long().clamp_(max=j - 1)]
    return bits[req, place].contiguous()


def prepare(case, seed):
    op = case["op"]
    s = {"op": op, "case": dict(case)}
    g = _gen(seed, 5)
    B, H, D = case["B"], case["Hkv"], case["D"]
    turn = torch.randperm(B, generator=g, device="cuda").tolist()
    if op == "attn":
        contexts, counts = ([v[i] for i in turn] for v in (_contexts(case), _row_counts(case)))
        s.update(_make_cache(g, case, [c + n for c, n in zip(contexts, counts)]))
        s["base"] = _i32(contexts)
        req, place = _places(counts)
        s["req"], s["place"] = req, place
        s["offsets"] = torch.cat([_i32([0]), torch.cumsum(_i32(counts), 0).to(torch.int32)])
        N, Hq = req.numel(), case["Hq"]
        qkv = (2.0 * _randn(g, max(N, 1), (Hq + 2 * H) * D)).to(torch.bfloat16)  # a fused projection's rows
        s["q"] = qkv[:N, :Hq * D].view(N, Hq, D)
        s["tree"] = _random_tree(g, req, place) if case["tree"] else None
        s["scale"] = D ** -0.5
        s["out"] = torch.empty((N, Hq, D), dtype=torch.bfloat16, device="cuda")
        if own:
            from draft_sampling_lossless_markov_gb300 import torch_api as T
            s["ws"] = T.tree_attention_workspace(B, case["rows"], Hq, H, D)
    else:
        R = case["rows"]
        if op == "move":
            contexts = [(r * 37) % 500 for r in turn]
            s.update(_make_cache(g, case, [c + 64 for c in contexts]))
            counts = [_path_counts(case)[i] for i in turn]
            n = _i32(counts)
            # ascending nodes, the first the root; the others lie past the places they go to
            nodes = torch.rand((B, 64), generator=g, device="cuda")
            nodes[:, :R] = 2.0
            path = torch.sort(torch.argsort(nodes, 1)[:, :R], 1).values.to(torch.int32)
            path[:, 0] = 0
            s["path"], s["n_path"] = path.contiguous(), n
            s["base"] = _i32(contexts)
            s["to_req"], s["to_place"] = _places(counts)  # the paths as one list
            s["from_place"] = path.long()[s["to_req"], s["to_place"]]
        else:
            contexts = [(r * 37) % 500 if R < 500 else 0 for r in turn]
            s.update(_make_cache(g, case, [c + R for c in contexts]))
            s["base"] = _i32(contexts)
            req, place = _places([R] * B)
            s["mark_req"], s["mark_pos"] = req.to(torch.int32), place.to(torch.int32)
            N = B * R
            if op == "write":
                kv = _randn(g, N, 2 * H * D)
                kv[:, :H * D] *= torch.exp(0.5 * _randn(g, H * D))
                kv = kv.to(DTYPES[case["dtype"]])
                s["k_new"], s["v_new"] = kv[:, :H * D].view(N, H, D), kv[:, H * D:].view(N, H, D)
            else:
                s["out"] = tuple(torch.empty((N, H, D), dtype=DTYPES[case["dtype"]], device="cuda") for _ in range(2))
    if own:
        from draft_sampling_lossless_markov_gb300 import torch_api as T
        s["cache"] = T.KvCache(s["k"], s["v"], s["table"], s["k_scale"], s["v_scale"])
    return s


# --------------------------------------------------------------------------- the plain forms, in 32 bits
def _take(pool, page, slot):
    """pool[page, :, slot]: [..., heads, D] or [..., heads]."""
    if pool.dtype == torch.float8_e4m3fn:
        return pool.view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn)
    return pool[page, :, slot]


def _put(pool, page, slot, values):
    if pool.dtype == torch.float8_e4m3fn:
        pool, values = pool.view(torch.uint8), values.view(torch.uint8)
    pool[page, :, slot] = values


def _where_is(s, req, pos):
    return s["table"][req, pos // s["page"]].long(), pos % s["page"]


def _attn_plain(s):
    table, base, q, req, place = s["table"], s["base"].long(), s["q"], s["req"], s["place"]
    N, Hq, D = q.shape
    B, R, H = table.shape[0], s["case"]["rows"], s["k"].shape[1]
    G = Hq // H
    L = int(s["case"]["L"]) + R
    count = (s["offsets"][1:] - s["offsets"][:-1]).long()
    t = torch.arange(L, device=q.device)
    held = t < (base + count)[:, None]  # [B, L]
    page = table.long().gather(1, (t // s["page"]).clamp(max=table.shape[1] - 1).expand(B, L)).clamp(min=0)
    slot = (t % s["page"]).expand(B, L)
    qp = torch.zeros((B, R, H, G, D), dtype=torch.float32, device=q.device)
    qp[req, place] = q.float().view(N, H, G, D)
    seen = t < base[:, None]  # [B, L], of every row
    if s["tree"] is None:
        mine = (t >= base[:, None])[:, None] & (t <= (base[:, None] + torch.arange(R, device=q.device))[:, :, None])
    else:
        bits = torch.zeros((B, R), dtype=torch.int64, device=q.device)
        bits[req, place] = s["tree"]
        node = t - base[:, None]  # [B, L]
        mine = ((node >= 0) & (node < 64))[:, None] & (((bits[:, :, None] >> node.clamp(0, 63)[:, None]) & 1) == 1)
    seen = ((seen[:, None] | mine) & held[:, None])  # [B, R, L]
    k = _take(s["k"], page, slot).float()  # [B, L, H, D]
    if s["k_scale"] is not None:
        k *= _take(s["k_scale"], page, slot)[..., None]
    z = torch.matmul(qp.permute(0, 2, 1, 3, 4).reshape(B, H, R * G, D), k.permute(0, 2, 3, 1))  # [B, H, R G, L]
    del k
    z *= s["scale"]
    z = z.view(B, H, R, G, L).masked_fill_(~seen[:, None, :, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    z -= torch.where(m > -math.inf, m, torch.zeros_like(m))
    z.exp_()
    total = z.sum(-1, keepdim=True)
    v = _take(s["v"], page, slot).float()
    if s["v_scale"] is not None:
        v *= _take(s["v_scale"], page, slot)[..., None]
    v.masked_fill_(~held[:, :, None, None], 0.0)
    o = torch.matmul(z.view(B, H, R * G, L), v.permute(0, 2, 1, 3)).view(B, H, R, G, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    s["out"].copy_(o.permute(0, 2, 1, 3, 4)[req, place].reshape(N, Hq, D))
    return s["out"]


def _quantised(x):
    amax = x.abs().amax(-1).clamp(min=AMAX_MIN)
    q = (x * (E4M3_MAX / amax)[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q, amax / E4M3_MAX


def _held(s):
    return {n: s[n] for n in ("k", "v", "k_scale", "v_scale") if s[n] is not None}


def _write_plain(s):
    req, place = s["mark_req"].long(), s["mark_pos"].long()
    page, slot = _where_is(s, req, s["base"].long()[req] + place)
    if s["k_scale"] is None:
        _put(s["k"], page, slot, s["k_new"].to(torch.bfloat16))
        _put(s["v"], page, slot, s["v_new"].to(torch.bfloat16))
        return _held(s)
    qk, sk = _quantised(s["k_new"].float())
    qv, sv = _quantised(s["v_new"].float())
    _put(s["k"], page, slot, qk)
    _put(s["v"], page, slot, qv)
    _put(s["k_scale"], page, slot, sk)
    _put(s["v_scale"], page, slot, sv)
    return _held(s)


def _read_plain(s):
    req, place = s["mark_req"].long(), s["mark_pos"].long()
    page, slot = _where_is(s, req, s["base"].long()[req] + place)
    k, v = _take(s["k"], page, slot).float(), _take(s["v"], page, slot).float()
    if s["k_scale"] is not None:
        k *= _take(s["k_scale"], page, slot)[..., None]
        v *= _take(s["v_scale"], page, slot)[..., None]
    s["out"][0].copy_(k)
    s["out"][1].copy_(v)
    return s["out"]


def _move_plain(s):
    first = s["base"].long()[s["to_req"]]
    page, slot = _where_is(s, s["to_req"], first + s["from_place"])
    to_page, to_slot = _where_is(s, s["to_req"], first + s["to_place"])
    _put(s["k"], to_page, to_slot, _take(s["k"], page, slot))
    _put(s["v"], to_page, to_slot, _take(s["v"], page, slot))
    if s["k_scale"] is not None:
        _put(s["k_scale"], to_page, to_slot, _take(s["k_scale"], page, slot))
        _put(s["v_scale"], to_page, to_slot, _take(s["v_scale"], page, slot))
    return _held(s)


def run(s):
    op = s["op"]
    if own:
        from draft_sampling_lossless_markov_gb300 import torch_api as T
        if op == "attn":
            return T.tree_attention(s["ws"], s["cache"], s["q"], s["offsets"], s["base"], s["case"]["rows"], tree=s["tree"],
                                    scale=s["scale"], out=s["out"])
        if op == "write":
            T.cache_write(s["cache"], s["k_new"], s["v_new"], s["mark_req"], s["mark_pos"], base=s["base"])
            return _held(s)
        if op == "read":
            return T.cache_read(s["cache"], s["mark_req"], s["mark_pos"], base=s["base"], out=s["out"])
        T.cache_move(s["cache"], s["base"], s["path"], s["n_path"])
        return _held(s)
    return {"attn": _attn_plain, "write": _write_plain, "read": _read_plain, "move": _move_plain}[op](s)


# --------------------------------------------------------------------------- the definition, in 64 bits
def _e4m3(v):
    """The e4m3 value nearest to v (ties to even, at most 448), for float64 v."""
    a = v.abs()
    _, e = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), torch.clamp(e - 1, min=-6) - 3)
    return torch.copysign(torch.clamp(torch.round(a / step) * step, max=E4M3_MAX), v)


def _rows_of(s, name, r, positions):
    """Rows [len(positions), Hkv, D] of request r in 64 bits, page by page."""
    P = s["page"]
    pages = s["table"][r].long()[positions // P]
    x = s[name].view(torch.uint8)[pages, :, positions % P].view(s[name].dtype) if s[name].dtype == torch.float8_e4m3fn else \
        s[name][pages, :, positions % P]
    x = x.to(torch.float64)
    if s[name + "_scale"] is not None:
        x = x * s[name + "_scale"][pages, :, positions % P].to(torch.float64)[:, :, None]
    return x


def _exact_attn(s):
    N, Hq, D = s["q"].shape
    out = torch.zeros((N, Hq, D), dtype=torch.float64, device="cuda")
    off, base = s["offsets"].tolist(), s["base"].tolist()
    H = s["k"].shape[1]
    for r in range(len(base)):
        lo, hi = off[r], off[r + 1]
        if hi == lo:
            continue
        total = base[r] + hi - lo
        at = torch.arange(total, device="cuda")
        words = [2 ** (j + 1) - 1 for j in range(hi - lo)] if s["tree"] is None else [w % 2 ** 64 for w in s["tree"][lo:hi].tolist()]
        mine = torch.tensor([[bool(w >> t & 1) for t in range(hi - lo)] for w in words], device="cuda")
        see = torch.cat([torch.ones((hi - lo, base[r]), dtype=torch.bool, device="cuda"), mine], 1)
        k, v = _rows_of(s, "k", r, at), _rows_of(s, "v", r, at)
        for h in range(H):
            heads = range(h * (Hq // H), (h + 1) * (Hq // H))
            q = s["q"][lo:hi, heads.start:heads.stop].to(torch.float64)  # [n, G, D]
            z = s["scale"] * (q.reshape(-1, D) @ k[:, h].T).view(hi - lo, len(heads), total)
            z = torch.where(see[:, None], z, z.new_tensor(-math.inf))
            p = torch.softmax(z, -1)
            p = torch.where(see.any(1)[:, None, None], p, torch.zeros_like(p))
            out[lo:hi, heads.start:heads.stop] = (p.view(-1, total) @ v[:, h]).view(hi - lo, len(heads), D)
    return out


def _exact_state(s):
    return {n: (t.to(torch.float64) if n.endswith("scale") else t.float().double()) for n, t in _held(s).items()}


def _exact_write(s):
    out = _exact_state(s)
    req, place = s["mark_req"].long(), s["mark_pos"].long()
    pos = s["base"].long()[req] + place
    page, slot = s["table"][req, pos // s["page"]].long(), pos % s["page"]
    for n in ("k", "v"):
        x = s[n + "_new"].to(torch.float64)
        if s[n + "_scale"] is None:
            out[n][page, :, slot] = x.to(torch.bfloat16).to(torch.float64)
            continue
        amax = torch.maximum(x.abs().amax(-1), x.new_tensor(AMAX_MIN))
        out[n][page, :, slot] = _e4m3(x * (E4M3_MAX / amax)[..., None])
        out[n + "_scale"][page, :, slot] = amax / E4M3_MAX
    return out


def _exact_read(s):
    base, B, R = s["base"].tolist(), s["case"]["B"], s["case"]["rows"]
    return tuple(torch.cat([_rows_of(s, n, r, base[r] + torch.arange(R, device="cuda")) for r in range(B)]) for n in ("k", "v"))


def _exact_move(s):
    old, out, P = _exact_state(s), _exact_state(s), s["page"]
    base, n_path = s["base"].long(), s["n_path"].long()
    for i in range(s["path"].shape[1]):
        r = torch.nonzero(n_path > i)[:, 0]
        a, b = base[r] + s["path"][r, i].long(), base[r] + i
        for n in out:
            out[n][s["table"][r, b // P].long(), :, b % P] = old[n][s["table"][r, a // P].long(), :, a % P]
    return out


def exact(case, seed):
    return {"attn": _exact_attn, "write": _exact_write, "read": _exact_read, "move": _exact_move}[case["op"]](prepare(case, seed))


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, H, D = case["op"], case["Hkv"], case["D"]
    held = 2 * H * (D * CODE_BYTES[case["cache"]] + (4 if case["cache"] == "e4m3" else 0))  # of one token
    if op == "attn":
        contexts, counts = _contexts(case), _row_counts(case)
        tokens = sum(c + n for c, n in zip(contexts, counts) if n)
        pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(contexts, counts))
        return {"bytes": tokens * held + sum(counts) * (2 * case["Hq"] * D * 2 + (8 if case["tree"] else 0)) + 8 * case["B"],
                "flops": 4 * D * case["Hq"] * pairs}
    if op == "move":
        n = sum(_path_counts(case))
        return {"bytes": 2 * n * held + 4 * n + 8 * case["B"], "flops": 0}
    n = case["B"] * case["rows"]
    return {"bytes": n * (held + 2 * H * D * BYTES[case["dtype"]] + 8) + 4 * case["B"], "flops": 3 * n * 2 * H * D}
