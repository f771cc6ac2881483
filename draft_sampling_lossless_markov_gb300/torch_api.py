"""Torch-tensor front end of the C ABI: turns tensors into the C structs.

PyTorch only provides device memory and streams here.  Each function checks
that its tensors are contiguous CUDA tensors of the expected dtype, fills the C
struct with their addresses and calls the library; a non-OK status raises.
Output tensors may be passed in (`out=`) to avoid allocation in a timed loop.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import numpy as np
import torch

from . import capi


class DsparkError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = f"{fn} returned {capi.dspark_status_string(status)}"
        if status == capi.DSPARK_CUDA_ERROR:
            msg += f" (cudaError {capi.dspark_last_cuda_error()})"
        super().__init__(msg)
        self.status = status


def _check(fn: str, st: int):
    if st != capi.DSPARK_OK:
        raise DsparkError(fn, st)


_DT = {torch.bfloat16: capi.DSPARK_BF16, torch.float32: capi.DSPARK_F32}


def _ptr(t: Optional[torch.Tensor], dtype=None) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("dspark tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("dspark tensors must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"expected {dtype}, got {t.dtype}")
    return t.data_ptr()


# the address of the current stream without a Stream object around it (3 us less a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def dims(B, gamma, V, r, H, dtype) -> capi.dspark_dims:
    return capi.dspark_dims(int(B), int(gamma), int(V), int(r), int(H), _DT[dtype] if dtype in _DT else int(dtype))


@dataclass
class Workspace:
    buf: torch.Tensor

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()

    @property
    def nbytes(self) -> int:
        return self.buf.numel()

    @classmethod
    def create(cls, d: capi.dspark_dims, device="cuda", stream=None) -> "Workspace":
        st, n = capi.dspark_workspace_size(d)
        _check("dspark_workspace_size", st)
        buf = torch.empty(max(n, 256), dtype=torch.uint8, device=device)
        ws = cls(buf)
        _check("dspark_workspace_init", capi.dspark_workspace_init(ws.ptr, ws.nbytes, _stream(stream)))
        return ws

    def read_error(self, stream=None):
        st, code, detail = capi.dspark_read_error(self.ptr, _stream(stream))
        _check("dspark_read_error", st)
        return code, detail


def _draft_args(U, W1, W2, h, w, anchor, temp, req_id, seed, out, W_rnn, rows, want_pd_stat):
    B, G, V = U.shape
    r = W1.shape[1] if W1 is not None else 0
    H = h.shape[2] if h is not None else 0
    dt = U.dtype
    dev = U.device
    if out is None:
        out = dict(tokens=torch.empty((B, G), dtype=torch.int32, device=dev),
                   pd_tok=torch.empty((B, G), dtype=torch.float32, device=dev),
                   conf_logit=torch.empty((B, G), dtype=torch.float32, device=dev),
                   conf=torch.empty((B, G), dtype=torch.float32, device=dev))
        if rows:
            out["pd_rows"] = torch.empty((B, G, V), dtype=torch.float32, device=dev)
        if want_pd_stat or not rows:
            out["pd_stat"] = torch.empty((B, G, 2), dtype=torch.float32, device=dev)
    a = capi.dspark_draft_args()
    a.dims = dims(B, G, V, r, H, dt)
    a.U, a.W1, a.W2, a.h, a.w = _ptr(U, dt), _ptr(W1, dt), _ptr(W2, dt), _ptr(h, dt), _ptr(w, dt)
    a.anchor, a.temp = _ptr(anchor, torch.int32), _ptr(temp, torch.float32)
    a.req_id = _ptr(req_id, torch.int32)
    a.seed = int(seed)
    a.tokens, a.pd_rows = _ptr(out["tokens"], torch.int32), _ptr(out.get("pd_rows"), torch.float32)
    a.pd_stat = _ptr(out.get("pd_stat"), torch.float32)
    a.pd_tok, a.conf_logit = _ptr(out["pd_tok"], torch.float32), _ptr(out["conf_logit"], torch.float32)
    a.conf = _ptr(out["conf"], torch.float32)
    if W_rnn is not None:
        a.W_rnn, a.head = _ptr(W_rnn, dt), capi.DSPARK_HEAD_RNN
    return a, out


def draft_sample(ws: Workspace, U, W1, W2, h, w, anchor, temp, req_id, seed: int, out: Optional[dict] = None,
                 stream=None, W_rnn=None, rows: bool = True, want_pd_stat: bool = False) -> dict:
    """dspark_draft_sample; W_rnn [3r, 2r + H] (the dtype of U) selects the RNN head;
    rows=False draws without p_d rows (pd_stat [B, gamma, 2] is then returned)."""
    a, out = _draft_args(U, W1, W2, h, w, anchor, temp, req_id, seed, out, W_rnn, rows, want_pd_stat)
    _check("dspark_draft_sample", capi.dspark_draft_sample(a, ws.ptr, ws.nbytes, _stream(stream)))
    return out


def _sched_args(conf_logit, sts_temp, sps, anchor, tokens, mode, out, n_verify_host, want_surv, conf_logit_prev):
    B, G = conf_logit.shape
    dev = conf_logit.device
    cap = B * (1 + G)
    if out is None:
        out = dict(ell=torch.empty(B, dtype=torch.int32, device=dev),
                   offsets=torch.empty(B + 1, dtype=torch.int32, device=dev),
                   flat_tok=torch.empty(cap, dtype=torch.int32, device=dev),
                   mark_req=torch.empty(cap, dtype=torch.int32, device=dev),
                   mark_pos=torch.empty(cap, dtype=torch.int32, device=dev),
                   n_verify=torch.empty(1, dtype=torch.int32, device=dev),
                   theta_best=torch.empty(1, dtype=torch.float64, device=dev))
        if want_surv:
            out["surv"] = torch.empty((B, G), dtype=torch.float32, device=dev)
    if isinstance(sps, np.ndarray):
        sps = torch.from_numpy(np.ascontiguousarray(sps, dtype=np.float64)).to(dev)
    a = capi.dspark_sched_args()
    a.B, a.gamma, a.mode = B, G, int(mode)
    a.conf_logit, a.sts_temp = _ptr(conf_logit, torch.float32), _ptr(sts_temp, torch.float32)
    a.sps = _ptr(sps, torch.float64) if sps is not None else None
    a.anchor, a.tokens = _ptr(anchor, torch.int32), _ptr(tokens, torch.int32)
    a.ell, a.offsets = _ptr(out["ell"], torch.int32), _ptr(out["offsets"], torch.int32)
    a.flat_tok, a.mark_req = _ptr(out["flat_tok"], torch.int32), _ptr(out["mark_req"], torch.int32)
    a.mark_pos, a.n_verify = _ptr(out["mark_pos"], torch.int32), _ptr(out["n_verify"], torch.int32)
    a.theta_best = _ptr(out["theta_best"], torch.float64)
    a.n_verify_host = n_verify_host.data_ptr() if n_verify_host is not None else None
    a.surv = _ptr(out.get("surv"), torch.float32)
    a.conf_logit_prev = _ptr(conf_logit_prev, torch.float32) if conf_logit_prev is not None else None
    out["_sps"] = sps  # keep the table alive while the call is in flight
    return a, out


def schedule(ws: Workspace, conf_logit, sts_temp, sps, anchor, tokens, mode: int, out: Optional[dict] = None,
             stream=None, n_verify_host: Optional[torch.Tensor] = None, want_surv=False,
             conf_logit_prev=None) -> dict:
    a, out = _sched_args(conf_logit, sts_temp, sps, anchor, tokens, mode, out, n_verify_host, want_surv,
                         conf_logit_prev)
    _check("dspark_schedule", capi.dspark_schedule(a, ws.ptr, ws.nbytes, _stream(stream)))
    return out


def draft_and_schedule(ws: Workspace, U, W1, W2, h, w, anchor, temp, req_id, seed: int, sts_temp, sps, mode: int,
                       out: Optional[dict] = None, sched_out: Optional[dict] = None, stream=None, W_rnn=None,
                       rows: bool = True, want_pd_stat: bool = False, n_verify_host: Optional[torch.Tensor] = None,
                       want_surv=False, conf_logit_prev=None) -> tuple:
    """dspark_draft_and_schedule: draft_sample then schedule of its confidences
    and tokens, in one call that may overlap them; returns (draft out, schedule out)."""
    da, out = _draft_args(U, W1, W2, h, w, anchor, temp, req_id, seed, out, W_rnn, rows, want_pd_stat)
    sa, sched_out = _sched_args(out["conf_logit"], sts_temp, sps, anchor, out["tokens"], mode, sched_out,
                                n_verify_host, want_surv, conf_logit_prev)
    _check("dspark_draft_and_schedule",
           capi.dspark_draft_and_schedule(da, sa, ws.ptr, ws.nbytes, _stream(stream)))
    return out, sched_out


def verify(ws: Workspace, target_logits, offsets, ell, tokens, pd_rows, pd_tok, temp, req_id, seed: int,
           out: Optional[dict] = None, stream=None, commit_cap=None, rejection: Optional[dict] = None) -> dict:
    """dspark_verify; commit_cap [B] i32 (the scheduled windows) selects cap-accept;
    rejection=dict(U, W1, W2, anchor, pd_stat) draws the residual by rejection
    from p_t (pd_rows may then be None)."""
    B, G = tokens.shape
    V = target_logits.shape[-1]
    dev = tokens.device
    dt = target_logits.dtype
    if out is None:
        out = dict(n_accept=torch.empty(B, dtype=torch.int32, device=dev),
                   out_tok=torch.empty((B, G + 1), dtype=torch.int32, device=dev),
                   n_out=torch.empty(B, dtype=torch.int32, device=dev))
    a = capi.dspark_verify_args()
    a.dims = dims(B, G, V, rejection["W1"].shape[1] if rejection else 0, 0, dt)
    a.target_logits = _ptr(target_logits, dt)
    a.offsets, a.ell, a.tokens = _ptr(offsets, torch.int32), _ptr(ell, torch.int32), _ptr(tokens, torch.int32)
    a.pd_rows, a.pd_tok = _ptr(pd_rows, torch.float32), _ptr(pd_tok, torch.float32)
    a.temp, a.req_id = _ptr(temp, torch.float32), _ptr(req_id, torch.int32)
    if rejection is not None:
        a.residual_mode = capi.DSPARK_RESIDUAL_REJECTION
        a.U, a.W1, a.W2 = _ptr(rejection["U"], dt), _ptr(rejection["W1"], dt), _ptr(rejection["W2"], dt)
        a.anchor, a.pd_stat = _ptr(rejection["anchor"], torch.int32), _ptr(rejection["pd_stat"], torch.float32)
    a.seed = int(seed)
    a.n_accept, a.out_tok, a.n_out = (_ptr(out["n_accept"], torch.int32), _ptr(out["out_tok"], torch.int32),
                                      _ptr(out["n_out"], torch.int32))
    a.commit_cap = _ptr(commit_cap, torch.int32) if commit_cap is not None else None
    _check("dspark_verify", capi.dspark_verify(a, ws.ptr, ws.nbytes, _stream(stream)))
    return out


def sts_fit_workspace(N: int, gamma: int, n_grid: int, n_bins: int, device="cuda", stream=None) -> Workspace:
    """Workspace of dspark_sts_fit (separate from the step workspace)."""
    st, n = capi.dspark_sts_fit_workspace_size(int(N), int(gamma), int(n_grid), int(n_bins))
    _check("dspark_sts_fit_workspace_size", st)
    ws = Workspace(torch.empty(max(n, 256), dtype=torch.uint8, device=device))
    _check("dspark_workspace_init", capi.dspark_workspace_init(ws.ptr, ws.nbytes, _stream(stream)))
    return ws


def sts_fit(ws: Workspace, conf_logit, accept_len, grid, n_bins: int, out: Optional[dict] = None, stream=None):
    """dspark_sts_fit: conf_logit [N, gamma] f32, accept_len [N] i32, grid [G] f32.
    Returns dict(sts_temp [gamma] f32, grid_index [gamma] i32, ece [gamma, G] f64)."""
    N, G = conf_logit.shape
    n_grid = grid.numel()
    dev = conf_logit.device
    if out is None:
        out = dict(sts_temp=torch.empty(G, dtype=torch.float32, device=dev),
                   grid_index=torch.empty(G, dtype=torch.int32, device=dev),
                   ece=torch.empty((G, n_grid), dtype=torch.float64, device=dev))
    a = capi.dspark_sts_fit_args()
    a.N, a.gamma, a.n_grid, a.n_bins = int(N), int(G), int(n_grid), int(n_bins)
    a.conf_logit = _ptr(conf_logit, torch.float32)
    a.accept_len = _ptr(accept_len, torch.int32)
    a.grid = _ptr(grid, torch.float32)
    a.sts_temp = _ptr(out["sts_temp"], torch.float32)
    a.grid_index = _ptr(out.get("grid_index"), torch.int32)
    a.ece = _ptr(out["ece"], torch.float64)
    _check("dspark_sts_fit", capi.dspark_sts_fit(a, ws.ptr, ws.nbytes, _stream(stream)))
    return out


def pack_rows(src, mark_req, mark_pos, n_rows, dst, ws: Optional[Workspace] = None, stream=None):
    """dspark_pack_rows: dst[i] = src[mark_req[i], mark_pos[i]] for i < n_rows[0].

    src [R, rows_per_request, V]: a CUDA tensor or a pinned CPU tensor (read by
    the GPU in place); mark_req, mark_pos [max_rows] and n_rows [1] int32 CUDA
    tensors; dst [max_rows, V] CUDA tensor of src's dtype."""
    if not src.is_contiguous() or not (src.is_cuda or src.is_pinned()):
        raise ValueError("src must be a contiguous CUDA tensor or a pinned CPU tensor")
    if src.dtype != dst.dtype:
        raise TypeError("src and dst dtypes differ")
    R, G1, V = src.shape
    a = capi.dspark_pack_args()
    a.V, a.dtype, a.rows_per_request, a.max_rows = int(V), _DT[src.dtype], int(G1), int(dst.shape[0])
    a.n_src_rows = int(R * G1)
    a.src = src.data_ptr()
    a.mark_req, a.mark_pos = _ptr(mark_req, torch.int32), _ptr(mark_pos, torch.int32)
    a.n_rows, a.dst = _ptr(n_rows, torch.int32), _ptr(dst)
    _check("dspark_pack_rows", capi.dspark_pack_rows(a, ws.ptr if ws is not None else 0, _stream(stream)))
    return dst


# ---------------------------------------------------------------------------
# The vocabulary projection and the answers around verify
# ---------------------------------------------------------------------------
def _rows(t: torch.Tensor, what: str, dtype) -> tuple:
    """(address, row stride in elements, rows, columns) of a 2-D CUDA tensor whose rows are dense."""
    if not t.is_cuda:
        raise ValueError("dspark tensors must live on a CUDA device")
    if t.dtype is not dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what} must be a 2-D tensor with dense rows")
    (rows, cols), (ld, step) = shape, t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{what} must be a 2-D tensor with dense rows")
    return t.data_ptr(), ld if rows > 1 else max(ld, cols), rows, cols


def _dense(t: Optional[torch.Tensor], shape: tuple, what: str, dtype) -> int:
    """The address of a dense CUDA tensor of this shape and type; 0 for None."""
    if t is None:
        return 0
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {shape}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what}: dspark tensors must be contiguous and live on a CUDA device")
    return t.data_ptr()


def _io_dtype(t: torch.Tensor, what: str) -> int:
    dt = _DT.get(t.dtype)
    if dt is None:
        raise TypeError(f"{what}: expected bfloat16 or float32, got {t.dtype}")
    return dt


_FP8 = torch.float8_e4m3fn


def fp8_codes(rows: int, cols: int, device="cuda") -> torch.Tensor:
    """An e4m3 matrix [rows, cols] whose row stride is the multiple of 16 bytes that matmul_fp8 needs."""
    return torch.empty((rows, -(-cols // 16) * 16), dtype=_FP8, device=device)[:, :cols]


def quant_fp8(x, block_rows: int = 1, out: Optional[tuple] = None, stream=None) -> tuple:
    """dspark_quant_fp8: x [M, K] (bf16 or f32, dense rows) to (codes [M, K] e4m3, scale
    [ceil(M / block_rows), ceil(K / 128)] f32); block_rows 1 for activations, 128 for weights."""
    dt = _io_dtype(x, "x")
    px, ldx, M, K = _rows(x, "x", x.dtype)
    if block_rows not in (1, 128):
        raise ValueError("block_rows is 1 or 128")
    shape = (-(-M // block_rows), -(-K // 128))
    if out is None:
        out = fp8_codes(M, K, x.device), torch.empty(shape, dtype=torch.float32, device=x.device)
    codes, scale = out
    pq, ldq, *got = _rows(codes, "codes", _FP8)
    if got != [M, K]:
        raise ValueError(f"codes: expected shape {(M, K)}, got {tuple(codes.shape)}")
    a = capi.pack_quant_fp8(M, K, dt, block_rows, px, ldx, pq, ldq, _dense(scale, shape, "scale", torch.float32))
    _check("dspark_quant_fp8", capi.dspark_quant_fp8(a, _stream(stream)))
    return out


def matmul_fp8_workspace(M: int, N: int, K: int, device="cuda", stream=None) -> Workspace:
    """Workspace of dspark_matmul_fp8 for products up to these sizes."""
    st, n = capi.dspark_matmul_fp8_workspace_size(int(M), int(N), int(K))
    _check("dspark_matmul_fp8_workspace_size", st)
    ws = Workspace(torch.empty(max(n, 256), dtype=torch.uint8, device=device))
    _check("dspark_workspace_init", capi.dspark_workspace_init(ws.ptr, ws.nbytes, _stream(stream)))
    return ws


def matmul_fp8(ws: Workspace, a, a_scale, w, w_scale, out=None, out_dtype=torch.bfloat16, n_rows=None, stream=None):
    """dspark_matmul_fp8: out [M, N] = (a a_scale) (w w_scale)^T for e4m3 a [M, K] and w [N, K] with a scale for each
    block of 128 (quant_fp8 with block_rows 1 and 128); n_rows [1] i32 bounds the rows computed."""
    pa, lda, M, K = _rows(a, "a", _FP8)
    pw, ldw, N, cols = _rows(w, "w", _FP8)
    if cols != K:
        raise ValueError(f"w: expected shape {(N, K)}, got {tuple(w.shape)}")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    dt = _io_dtype(out, "out")
    po, ldo, *got = _rows(out, "out", out.dtype)
    if got != [M, N]:
        raise ValueError(f"out: expected shape {(M, N)}, got {tuple(out.shape)}")
    kb, f32 = -(-K // 128), torch.float32
    c = capi.pack_matmul_fp8(M, N, K, dt, pa, lda, _dense(a_scale, (M, kb), "a_scale", f32), pw, ldw,
                             _dense(w_scale, (-(-N // 128), kb), "w_scale", f32), po, ldo,
                             _dense(n_rows, (1,), "n_rows", torch.int32))
    _check("dspark_matmul_fp8", capi.dspark_matmul_fp8(c, ws.ptr, ws.nbytes, _stream(stream)))
    return out


def _logit_rows(logits, tokens, temp, mask, mark_req, mark_pos, n_rows) -> tuple:
    """The values of a dspark_logit_rows."""
    dt = _io_dtype(logits, "logits")
    p, ld, N, V = _rows(logits, "logits", logits.dtype)
    i32, f32 = torch.int32, torch.float32
    if mark_req is None and mark_pos is None:
        n_req = cols = 0
        pt, pT = _dense(tokens, (N,), "tokens", i32), _dense(temp, (N,), "temp", f32)
    else:
        if mark_req is None or mark_pos is None:
            raise ValueError("mark_req and mark_pos go together")
        if tokens.dim() != 2:
            raise ValueError("tokens [n_req, tok_cols] is needed with markers")
        n_req, cols = tokens.shape
        pt, pT = _dense(tokens, (n_req, cols), "tokens", i32), _dense(temp, (n_req,), "temp", f32)
    pm = ldm = 0
    if mask is not None:
        pm, ldm, mask_rows, words = _rows(mask, "mask", i32)
        if mask_rows != N or words < -(-V // 32):
            raise ValueError("mask: expected [N, >= ceil(V / 32)] words")
    return (N, V, dt, cols, n_req, p, ld, pt, pT, pm, ldm, _dense(mark_req, (N,), "mark_req", i32),
            _dense(mark_pos, (N,), "mark_pos", i32), _dense(n_rows, (1,), "n_rows", i32))


def token_logprobs_workspace(N: int, V: int, top: int, device="cuda", stream=None) -> Workspace:
    """Workspace of dspark_token_logprobs for up to these sizes."""
    st, n = capi.dspark_token_logprobs_workspace_size(int(N), int(V), int(top))
    _check("dspark_token_logprobs_workspace_size", st)
    ws = Workspace(torch.empty(max(n, 256), dtype=torch.uint8, device=device))
    _check("dspark_workspace_init", capi.dspark_workspace_init(ws.ptr, ws.nbytes, _stream(stream)))
    return ws


def token_logprobs(ws: Workspace, logits, tokens, temp=None, top: int = 0, mask=None, mark_req=None, mark_pos=None,
                   n_rows=None, out: Optional[dict] = None, stream=None) -> dict:
    """dspark_token_logprobs: per row of logits [N, V] the log probability and rank of its token, the entropy, the
    first `top` alternatives and the statistics its gradient needs.  tokens [N] i32 and temp [N] f32, or with markers
    tokens [n_req, tok_cols] and temp [n_req]; mask [N, >= ceil(V / 32)] i32 holds a bit a place.
    Returns dict(logprob, entropy, rank, row_stat, top_id, top_logprob); an `out` may leave keys out (top_id and
    top_logprob only when top is 0)."""
    rows = _logit_rows(logits, tokens, temp, mask, mark_req, mark_pos, n_rows)
    N = rows[0]
    f32, i32 = torch.float32, torch.int32
    if out is None:
        new = lambda shape, dt: torch.empty(shape, dtype=dt, device=logits.device)  # noqa: E731
        out = dict(logprob=new(N, f32), entropy=new(N, f32), rank=new(N, i32), row_stat=new((N, 2), f32),
                   top_id=new((N, top), i32), top_logprob=new((N, top), f32))
    get = out.get
    a = capi.pack_token_logprobs(
        *rows, top, _dense(get("logprob"), (N,), "logprob", f32), _dense(get("entropy"), (N,), "entropy", f32),
        _dense(get("rank"), (N,), "rank", i32), _dense(get("row_stat"), (N, 2), "row_stat", f32),
        _dense(get("top_id"), (N, top), "top_id", i32), _dense(get("top_logprob"), (N, top), "top_logprob", f32))
    _check("dspark_token_logprobs", capi.dspark_token_logprobs(a, ws.ptr, ws.nbytes, _stream(stream)))
    return out


def token_logprobs_grad(ws: Optional[Workspace], logits, tokens, row_stat, entropy=None, top_id=None, g_logprob=None,
                        g_entropy=None, g_top=None, temp=None, mask=None, mark_req=None, mark_pos=None, n_rows=None,
                        out=None, stream=None):
    """dspark_token_logprobs_grad: the gradient by the logits of sum(g_logprob logprob) + sum(g_entropy entropy) +
    sum(g_top top_logprob), from token_logprobs's row_stat, entropy and top_id.  out may be logits itself."""
    rows = _logit_rows(logits, tokens, temp, mask, mark_req, mark_pos, n_rows)
    N, V = rows[:2]
    f32 = torch.float32
    top = 0
    if g_top is not None:
        if top_id is None:
            raise ValueError("g_top needs top_id")
        if g_top.dim() != 2:
            raise ValueError("g_top: expected [N, top]")
        top = g_top.shape[1]
    if g_entropy is not None and entropy is None:
        raise ValueError("g_entropy needs entropy")
    if out is None:
        out = torch.empty((N, V), dtype=logits.dtype, device=logits.device)
    po, ldo, *got = _rows(out, "out", logits.dtype)
    if got != [N, V]:
        raise ValueError(f"out: expected shape {(N, V)}, got {tuple(out.shape)}")
    a = capi.pack_token_logprobs_grad(
        *rows, top, _dense(row_stat, (N, 2), "row_stat", f32),
        _dense(entropy, (N,), "entropy", f32) if g_entropy is not None else 0,
        _dense(top_id, (N, top), "top_id", torch.int32) if top else 0, _dense(g_logprob, (N,), "g_logprob", f32),
        _dense(g_entropy, (N,), "g_entropy", f32), _dense(g_top, (N, top), "g_top", f32) if top else 0, po, ldo)
    _check("dspark_token_logprobs_grad",
           capi.dspark_token_logprobs_grad(a, ws.ptr if ws is not None else 0, _stream(stream)))
    return out


# ---------------------------------------------------------------------------
# The key/value cache and the attention of a step's drafted rows
# ---------------------------------------------------------------------------
class KvCache:
    """dspark_kv_cache: k and v [n_pages, n_kv_heads, page_size, head_dim] (e4m3 with k_scale and v_scale [n_pages,
    n_kv_heads, page_size] f32, or bf16 without), table [n_req, max_pages] i32 (dense rows).  The tensors are checked
    here, once; the calls write into them.  Their contents may change (a table's entries in place), the tensors may not."""

    def __setattr__(self, name, value):
        if "fields" in self.__dict__:  # the calls would go on with the addresses of the old tensor
            raise AttributeError(f"{name}: a KvCache keeps its tensors, make another for others")
        super().__setattr__(name, value)

    def __init__(self, k, v, table, k_scale=None, v_scale=None):
        if k.dim() != 4:
            raise ValueError("k must be [n_pages, n_kv_heads, page_size, head_dim]")
        shape = tuple(k.shape)
        if k.dtype is _FP8:
            dt = capi.DSPARK_E4M3
            if k_scale is None or v_scale is None:
                raise ValueError("an e4m3 cache needs k_scale and v_scale")
        elif k.dtype is torch.bfloat16:
            dt = capi.DSPARK_BF16
            if k_scale is not None or v_scale is not None:
                raise ValueError("a bf16 cache has no scales")
        else:
            raise TypeError(f"k: expected float8_e4m3fn or bfloat16, got {k.dtype}")
        pt, ldt, n_req, max_pages = _rows(table, "table", torch.int32)
        n_pages, heads, page, dim = shape
        f32 = torch.float32
        self.k, self.v, self.k_scale, self.v_scale, self.table = k, v, k_scale, v_scale, table
        self.n_kv_heads, self.head_dim, self.n_req = heads, dim, n_req
        self.fields = (n_pages, page, heads, dim, dt, n_req, max_pages, _dense(k, shape, "k", k.dtype),
                       _dense(v, shape, "v", k.dtype), _dense(k_scale, shape[:3], "k_scale", f32),
                       _dense(v_scale, shape[:3], "v_scale", f32), pt, ldt)

    @classmethod
    def create(cls, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, table, dtype=_FP8) -> "KvCache":
        """A cache of zeros."""
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        new = [torch.zeros(shape, dtype=torch.uint8 if dtype is _FP8 else dtype, device=table.device) for _ in range(2)]
        if dtype is not _FP8:
            return cls(*new, table)
        scales = [torch.zeros(shape[:3], dtype=torch.float32, device=table.device) for _ in range(2)]
        return cls(*(t.view(_FP8) for t in new), table, *scales)


def _heads(t: torch.Tensor, what: str, dtype) -> tuple:
    """(address, row stride in elements, rows, heads, head size) of a 3-D CUDA tensor whose rows are dense."""
    if not t.is_cuda:
        raise ValueError("dspark tensors must live on a CUDA device")
    if t.dtype is not dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{what} must be a 3-D tensor with dense rows")
    (rows, heads, dim), (ld, per_head, step) = shape, t.stride()
    if (step != 1 and dim > 1) or (per_head != dim and heads > 1):
        raise ValueError(f"{what} must be a 3-D tensor with dense rows")
    return t.data_ptr(), ld if rows > 1 else max(ld, heads * dim), rows, heads, dim


def _cache_rows(cache: KvCache, k, v, mark_req, mark_pos, base, n_rows) -> tuple:
    """The values of a cache write or read."""
    dt = _io_dtype(k, "k")
    pk, ldk, N, *got = _heads(k, "k", k.dtype)
    if got != [cache.n_kv_heads, cache.head_dim]:
        raise ValueError(f"k: expected [N, {cache.n_kv_heads}, {cache.head_dim}], got {tuple(k.shape)}")
    if v.shape != k.shape:
        raise ValueError(f"v: expected shape {tuple(k.shape)}, got {tuple(v.shape)}")
    if v.dtype is k.dtype and v.is_cuda and v.stride() == k.stride():
        pv, ldv = v.data_ptr(), ldk  # laid out as k
    else:
        pv, ldv, *got = _heads(v, "v", k.dtype)
    i32 = torch.int32
    return (*cache.fields, N, dt, pk, ldk, pv, ldv, _dense(mark_req, (N,), "mark_req", i32),
            _dense(mark_pos, (N,), "mark_pos", i32), _dense(base, (cache.n_req,), "base", i32),
            _dense(n_rows, (1,), "n_rows", i32))


def cache_write(cache: KvCache, k, v, mark_req, mark_pos, base=None, n_rows=None, ws: Optional[Workspace] = None,
                stream=None) -> None:
    """dspark_cache_write: rows k, v [N, n_kv_heads, head_dim] (bf16 or f32, dense rows) go to request mark_req[i],
    position base[mark_req[i]] + mark_pos[i]; mark_req -1 skips a row; ws takes the errors, if given."""
    a = capi.pack_cache_write(*_cache_rows(cache, k, v, mark_req, mark_pos, base, n_rows))
    _check("dspark_cache_write", capi.dspark_cache_write(a, ws.ptr if ws is not None else 0, _stream(stream)))


def cache_read(cache: KvCache, mark_req, mark_pos, base=None, n_rows=None, out: Optional[tuple] = None,
               dtype=torch.bfloat16, ws: Optional[Workspace] = None, stream=None) -> tuple:
    """dspark_cache_read: (k, v) [N, n_kv_heads, head_dim] of such places, in `dtype` or the type of `out`."""
    if out is None:
        shape = (mark_req.numel(), cache.n_kv_heads, cache.head_dim)
        out = tuple(torch.empty(shape, dtype=dtype, device=cache.k.device) for _ in range(2))
    a = capi.pack_cache_read(*_cache_rows(cache, out[0], out[1], mark_req, mark_pos, base, n_rows))
    _check("dspark_cache_read", capi.dspark_cache_read(a, ws.ptr if ws is not None else 0, _stream(stream)))
    return out


def cache_move(cache: KvCache, base, path, n_path, ws: Optional[Workspace] = None, stream=None) -> None:
    """dspark_cache_move: position base[r] + i takes what base[r] + path[r, i] held, for i < n_path[r]; path [n_req,
    path_cols] i32 (dense rows), base and n_path [n_req] i32."""
    i32 = torch.int32
    pp, ldp, rows, cols = _rows(path, "path", i32)
    if rows != cache.n_req:
        raise ValueError(f"path: expected {cache.n_req} rows, got {rows}")
    a = capi.pack_cache_move(*cache.fields, cols, _dense(base, (rows,), "base", i32), pp, ldp,
                             _dense(n_path, (rows,), "n_path", i32))
    _check("dspark_cache_move", capi.dspark_cache_move(a, ws.ptr if ws is not None else 0, _stream(stream)))


def tree_attention_workspace(n_req: int, max_tree: int, n_q_heads: int, n_kv_heads: int, head_dim: int, device="cuda",
                             stream=None) -> Workspace:
    """Workspace of dspark_tree_attention for up to these sizes."""
    st, n = capi.dspark_tree_attention_workspace_size(int(n_req), int(max_tree), int(n_q_heads), int(n_kv_heads),
                                                      int(head_dim))
    _check("dspark_tree_attention_workspace_size", st)
    ws = Workspace(torch.empty(max(n, 256), dtype=torch.uint8, device=device))
    _check("dspark_workspace_init", capi.dspark_workspace_init(ws.ptr, ws.nbytes, _stream(stream)))
    return ws


def tree_attention(ws: Workspace, cache: KvCache, q, offsets, base, max_tree: int, tree=None, scale: Optional[float] = None,
                   out=None, stream=None):
    """dspark_tree_attention: rows offsets[r] .. offsets[r + 1] - 1 of q [N, n_q_heads, head_dim] (bf16, dense rows), at
    most max_tree of them, attend to request r's first base[r] cached positions and to the drafted rows behind them that
    tree [N] i64 (bit t: the request's row t) shows, all up to themselves without a tree.  scale: head_dim ** -0.5."""
    bf16, i32 = torch.bfloat16, torch.int32
    pq, ldq, N, heads, dim = _heads(q, "q", bf16)
    if dim != cache.head_dim:
        raise ValueError(f"q: expected head size {cache.head_dim}, got {dim}")
    if out is None:
        out = torch.empty((N, heads, dim), dtype=bf16, device=q.device)
    po, ldo, *got = _heads(out, "out", bf16)
    if got != [N, heads, dim]:
        raise ValueError(f"out: expected shape {(N, heads, dim)}, got {tuple(out.shape)}")
    a = capi.pack_tree_attention(*cache.fields, N, heads, max_tree, dim ** -0.5 if scale is None else scale, pq, ldq, po, ldo,
                                 _dense(offsets, (cache.n_req + 1,), "offsets", i32),
                                 _dense(base, (cache.n_req,), "base", i32), _dense(tree, (N,), "tree", torch.int64))
    _check("dspark_tree_attention", capi.dspark_tree_attention(a, ws.ptr, ws.nbytes, _stream(stream)))
    return out
