// C ABI of the dspark library: argument checks, workspace layout, dispatch.
// Every check happens before anything is enqueued; nothing here allocates.
#include <algorithm>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <atomic>
#include <map>
#include <mutex>
#include <utility>

#include "common.cuh"
#include "dspark.h"
#include "internal.h"

namespace dspark {

size_t elem_size(int dtype) { return dtype == DSPARK_BF16 ? 2 : 4; }

static std::atomic<uint64_t> g_launches{0};
void count_launches(int n) { g_launches.fetch_add((uint64_t)n, std::memory_order_relaxed); }

static bool dims_ok(const dspark_dims& d) {
  if (d.B < 0 || d.gamma < 1 || d.gamma > DSPARK_MAX_GAMMA || d.V < 1 || d.V > DSPARK_MAX_VOCAB) return false;
  if (d.r < 0 || d.r > DSPARK_MAX_RANK || d.H < 0) return false;
  if (d.dtype != DSPARK_BF16 && d.dtype != DSPARK_F32) return false;
  // index arithmetic stays in 64 bits; per-row sizes must fit in 32 bits
  if ((int64_t)d.B * (d.gamma + 1) > (int64_t)INT32_MAX) return false;
  return true;
}

WsLayout ws_layout(const dspark_dims& d) {
  WsLayout L;
  const size_t B = (size_t)d.B, G = (size_t)d.gamma, V = (size_t)d.V, r = (size_t)d.r;
  size_t off = sizeof(WsHeader);
  auto take = [&](size_t bytes) {
    off = align_up(off, 256);
    const size_t at = off;
    off += bytes;
    return at;
  };
  // regions that depend on (B, gamma) only come first, so that dspark_schedule
  // and dspark_verify find them at the same offsets whatever V, r, H and dtype
  L.sk0 = take(B * G * sizeof(uint32_t));
  L.sk1 = take(B * G * sizeof(uint32_t));
  L.sv0 = take(B * G * sizeof(uint32_t));
  L.sv1 = take(B * G * sizeof(uint32_t));
  L.vrs = take(B * (G + 1) * RS_PARTS * sizeof(float4));
  L.vm = take(B * sizeof(int32_t));
  L.vrowT = take(B * (G + 1) * sizeof(float));
  L.vfmeta = take(B * 4 * sizeof(int32_t));
  L.vfstat = take(B * 4 * sizeof(float));
  L.zh = take(B * G * sizeof(float));
  L.rowstat = take(B * sizeof(float2));
  L.sel = take(B * sizeof(float4));
  // two buffers, positions alternate; fp32-sized so that the RNN head's computed
  // rows fit whatever the dtype
  L.E = take(2 * B * r * sizeof(float));
  L.rnn_s = take(2 * B * r * sizeof(float));  // RNN head state s_{k-1}, s_k
  L.rnn_p = take(B * G * 3 * r * sizeof(float));  // RNN head: W_rnn[:, 2r:] . h_k of every position
  L.rnn_z = take(B * 4 * r * sizeof(uint16_t));     // RNN head, tensor-core recurrent step: z''
  L.rnn_wz = take(3 * r * 4 * r * sizeof(uint16_t));  // its packed weights
  L.rnn_pre = take(B * 3 * r * sizeof(float));      // its products
  const size_t ntiles = (V + kPartialTileMin - 1) / kPartialTileMin;
  // (the fused draft kernel keeps float2 partials of 64-column chunks, rows
  // padded to a multiple of 128)
  const size_t fused_row = ((V + 64 * 128 - 1) / (64 * 128)) * 128 * sizeof(float2);
  L.part = take(B * std::max(ntiles * sizeof(float4), fused_row));
  L.segpart = take(B * kDraftMaxSeg * sizeof(float4));
  // grid-barrier counter, then one tile counter per (sweep, M-tile) (gamma + 1
  // sweeps), then the RNN head's recurrent-unit counters per (position,
  // M-tile); all zeroed by one memset per draft call
  L.gbar = take(16 + (2 * G + 1) * ((B + 127) / 128) * sizeof(uint32_t));
  L.vfin = take(B * 32 * ((((V + 255) / 256) + 31) / 32) * sizeof(float2));
  L.total = align_up(off, 256);
  return L;
}

cudaError_t ensure_smem_limit(const void* func, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::mutex mu;
  static std::map<std::pair<int, const void*>, int> set_to;  // (device, kernel) -> limit set
  std::lock_guard<std::mutex> lock(mu);
  int& cur = set_to[std::make_pair(dev, func)];
  if (cur >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) cur = bytes;
  return e;
}

static bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

static dspark_status check_ws(const dspark_dims& d, void* ws, size_t bytes, WsLayout* L) {
  if (!ws || ((uintptr_t)ws & 255u)) return DSPARK_INVALID_ARG;
  *L = ws_layout(d);
  if (bytes < L->total) return DSPARK_INVALID_ARG;
  return DSPARK_OK;
}

// the CUDA error behind the last DSPARK_CUDA_ERROR returned on this thread
static thread_local int t_last_cuda_error = 0;

dspark_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return DSPARK_OK;
  t_last_cuda_error = (int)e;
  return DSPARK_CUDA_ERROR;
}

dspark_status check_sched_args(const dspark_sched_args* a, int64_t max_keys) {
  if (!a || a->B < 0 || a->gamma < 1 || a->gamma > DSPARK_MAX_GAMMA) return DSPARK_INVALID_ARG;
  if (a->mode != DSPARK_SCHED_OFF && a->mode != DSPARK_SCHED_GREEDY && a->mode != DSPARK_SCHED_ASYNC_TOPK)
    return DSPARK_INVALID_ARG;
  if ((int64_t)a->B * a->gamma > max_keys) return DSPARK_UNSUPPORTED;
  if (a->B == 0) return DSPARK_OK;
  if (!a->conf_logit || !a->sts_temp || !a->anchor || !a->tokens || !a->ell || !a->offsets || !a->flat_tok ||
      !a->mark_req || !a->mark_pos || !a->n_verify || !a->theta_best)
    return DSPARK_INVALID_ARG;
  if (a->mode != DSPARK_SCHED_OFF && !a->sps) return DSPARK_INVALID_ARG;
  if (a->mode == DSPARK_SCHED_ASYNC_TOPK) {
    if (!a->conf_logit_prev) return DSPARK_INVALID_ARG;
    if (!schedule_async_supported(a->B, a->gamma)) return DSPARK_UNSUPPORTED;
  }
  return DSPARK_OK;
}

}  // namespace dspark

using namespace dspark;

// sizes of the vocabulary calls whose tile counts and rounded-up lengths stay in 32 bits
constexpr int32_t kMaxVocabDim = 1 << 30;

// A launcher's result as a status; nothing it throws (a table that cannot grow)
// leaves the C entry.
template <typename F>
static dspark_status launched(F launch) {
  try {
    const cudaError_t e = launch();
    return e == cudaErrorNotSupported ? DSPARK_UNSUPPORTED : cuda_status(e);
  } catch (...) {
    return cuda_status(cudaErrorMemoryAllocation);
  }
}

extern "C" {

const char* dspark_status_string(dspark_status s) {
  switch (s) {
    case DSPARK_OK: return "DSPARK_OK";
    case DSPARK_INVALID_ARG: return "DSPARK_INVALID_ARG";
    case DSPARK_UNSUPPORTED: return "DSPARK_UNSUPPORTED";
    case DSPARK_CUDA_ERROR: return "DSPARK_CUDA_ERROR";
    case DSPARK_TIMEOUT: return "DSPARK_TIMEOUT";
    case DSPARK_BAD_INPUT: return "DSPARK_BAD_INPUT";
  }
  return "DSPARK_UNKNOWN_STATUS";
}

const char* dspark_version(void) { return "dspark-gb300 0.1 (sm_103a)"; }

uint64_t dspark_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

int dspark_last_cuda_error(void) { return t_last_cuda_error; }

dspark_status dspark_workspace_size(const dspark_dims* dims, size_t* bytes) {
  if (!dims || !bytes || !dims_ok(*dims)) return DSPARK_INVALID_ARG;
  *bytes = ws_layout(*dims).total;
  return DSPARK_OK;
}

dspark_status dspark_workspace_init(void* workspace, size_t workspace_bytes, void* stream) {
  if (!workspace || workspace_bytes < sizeof(WsHeader)) return DSPARK_INVALID_ARG;
  return cuda_status(cudaMemsetAsync(workspace, 0, sizeof(WsHeader), (cudaStream_t)stream));
}

dspark_status dspark_read_error(void* workspace, int32_t* code_host, int32_t* detail_host, void* stream) {
  if (!workspace || !code_host) return DSPARK_INVALID_ARG;
  WsHeader h;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = cudaMemcpyAsync(&h, workspace, 2 * sizeof(int32_t), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return DSPARK_CUDA_ERROR;
  *code_host = h.err_code;
  if (detail_host) *detail_host = h.err_detail;
  e = cudaMemsetAsync(workspace, 0, 2 * sizeof(int32_t), s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return cuda_status(e);
}

// The checks of dspark_draft_sample (B > 0), with the workspace layout.
static dspark_status check_draft_args(const dspark_draft_args* a, void* workspace, size_t workspace_bytes,
                                      WsLayout* L) {
  const dspark_dims& d = a->dims;
  if (!a->U || !a->anchor || !a->temp || !a->req_id || !a->tokens || !a->pd_tok || !a->conf_logit || !a->conf)
    return DSPARK_INVALID_ARG;
  if (!a->pd_rows && (!a->pd_stat || a->head != DSPARK_HEAD_MARKOV)) return DSPARK_INVALID_ARG;
  if (d.r > 0 && (!a->W1 || !a->W2)) return DSPARK_INVALID_ARG;
  if (d.H + d.r > 0 && !a->w) return DSPARK_INVALID_ARG;
  if (d.H > 0 && !a->h) return DSPARK_INVALID_ARG;
  if (a->head != DSPARK_HEAD_MARKOV && a->head != DSPARK_HEAD_RNN) return DSPARK_INVALID_ARG;
  if (a->head == DSPARK_HEAD_RNN && (d.r < 1 || !a->W_rnn)) return DSPARK_INVALID_ARG;
  const void* big[] = {a->U, a->W1, a->W2, a->h, a->w, a->pd_rows, a->head == DSPARK_HEAD_RNN ? a->W_rnn : nullptr};
  for (const void* p : big)
    if (p && !aligned16(p)) return DSPARK_INVALID_ARG;
  return check_ws(d, workspace, workspace_bytes, L);
}

dspark_status dspark_draft_sample(const dspark_draft_args* a, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  if (!a || !dims_ok(a->dims)) return DSPARK_INVALID_ARG;
  if (a->dims.B == 0) return DSPARK_OK;
  WsLayout L;
  const dspark_status st = check_draft_args(a, workspace, workspace_bytes, &L);
  if (st != DSPARK_OK) return st;
  const cudaError_t e = launch_draft(*a, static_cast<uint8_t*>(workspace), L, (cudaStream_t)stream);
  if (e == cudaErrorNotSupported && !a->pd_rows) return DSPARK_UNSUPPORTED;  // no fused path for the row-free mode
  return cuda_status(e);
}

dspark_status dspark_draft_and_schedule(const dspark_draft_args* da, const dspark_sched_args* sa, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  if (!da || !dims_ok(da->dims)) return DSPARK_INVALID_ARG;
  const dspark_status chk = check_sched_args(sa, DSPARK_MAX_SCHED_KEYS);
  if (chk != DSPARK_OK) return chk;
  // the schedule reads the draft's confidences and tokens
  if (sa->B != da->dims.B || sa->gamma != da->dims.gamma) return DSPARK_INVALID_ARG;
  if (da->dims.B == 0) return DSPARK_OK;
  if (sa->conf_logit != da->conf_logit || sa->tokens != da->tokens || sa->anchor != da->anchor)
    return DSPARK_INVALID_ARG;
  WsLayout L;
  const dspark_status st = check_draft_args(da, workspace, workspace_bytes, &L);
  if (st != DSPARK_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const cudaStream_t s = (cudaStream_t)stream;
  DraftOverlap ov;
  ov.want = schedule_behind_draft_supported(sa->B, sa->gamma);
  cudaError_t e = launch_draft(*da, ws, L, s, &ov);
  if (e == cudaErrorNotSupported && !da->pd_rows) return DSPARK_UNSUPPORTED;
  if (e != cudaSuccess) return cuda_status(e);
  e = ov.armed ? launch_schedule_behind_draft(*sa, ws, L, ov.sel_done, ov.n_ctas, s) : launch_schedule(*sa, ws, L, s);
  return cuda_status(e);
}

dspark_status dspark_schedule(const dspark_sched_args* a, void* workspace, size_t workspace_bytes, void* stream) {
  const dspark_status chk = check_sched_args(a, DSPARK_MAX_SCHED_KEYS);
  if (chk != DSPARK_OK || a->B == 0) return chk;
  dspark_dims d{a->B, a->gamma, 1, 0, 0, DSPARK_F32};
  WsLayout L;
  const dspark_status st = check_ws(d, workspace, workspace_bytes, &L);
  if (st != DSPARK_OK) return st;
  return cuda_status(launch_schedule(*a, static_cast<uint8_t*>(workspace), L, (cudaStream_t)stream));
}

dspark_status dspark_verify(const dspark_verify_args* a, void* workspace, size_t workspace_bytes, void* stream) {
  if (!a || !dims_ok(a->dims)) return DSPARK_INVALID_ARG;
  const dspark_dims& d = a->dims;
  if (d.B == 0) return DSPARK_OK;
  if (!a->target_logits || !a->offsets || !a->ell || !a->tokens || !a->pd_tok || !a->temp || !a->req_id ||
      !a->n_accept || !a->out_tok || !a->n_out)
    return DSPARK_INVALID_ARG;
  if (a->residual_mode != DSPARK_RESIDUAL_INVERSE_CDF && a->residual_mode != DSPARK_RESIDUAL_REJECTION)
    return DSPARK_INVALID_ARG;
  if (a->residual_mode == DSPARK_RESIDUAL_INVERSE_CDF && !a->pd_rows) return DSPARK_INVALID_ARG;
  if (a->residual_mode == DSPARK_RESIDUAL_REJECTION &&
      (d.r < 1 || !a->U || !a->W1 || !a->W2 || !a->anchor || !a->pd_stat))
    return DSPARK_INVALID_ARG;
  if (!aligned16(a->target_logits) || (a->pd_rows && !aligned16(a->pd_rows))) return DSPARK_INVALID_ARG;
  WsLayout L;
  const dspark_status st = check_ws(d, workspace, workspace_bytes, &L);
  if (st != DSPARK_OK) return st;
  return cuda_status(launch_verify(*a, static_cast<uint8_t*>(workspace), L, (cudaStream_t)stream));
}

dspark_status dspark_pack_rows(const dspark_pack_args* a, void* workspace, void* stream) {
  if (!a || a->V < 1 || a->V > DSPARK_MAX_VOCAB || (a->dtype != DSPARK_BF16 && a->dtype != DSPARK_F32)) return DSPARK_INVALID_ARG;
  if (a->rows_per_request < 1 || a->max_rows < 0 || a->n_src_rows < 0) return DSPARK_INVALID_ARG;
  if (a->max_rows == 0) return DSPARK_OK;
  if (!a->src || !a->mark_req || !a->mark_pos || !a->n_rows || !a->dst) return DSPARK_INVALID_ARG;
  if (workspace && ((uintptr_t)workspace & 255u)) return DSPARK_INVALID_ARG;
  return cuda_status(launch_pack_rows(*a, static_cast<WsHeader*>(workspace), (cudaStream_t)stream));
}

static bool sts_dims_ok(int32_t N, int32_t gamma, int32_t n_grid, int32_t n_bins) {
  if (N < 0 || N > DSPARK_STS_MAX_SAMPLES || gamma < 1 || gamma > DSPARK_MAX_GAMMA) return false;
  if (n_grid < 1 || n_bins < 1) return false;
  return (int64_t)n_bins * std::max<int32_t>(n_grid, 128) <= DSPARK_STS_MAX_TABLE;
}

dspark_status dspark_sts_fit_workspace_size(int32_t N, int32_t gamma, int32_t n_grid, int32_t n_bins,
                                            size_t* bytes) {
  if (!bytes || !sts_dims_ok(N, gamma, n_grid, n_bins)) return DSPARK_INVALID_ARG;
  *bytes = sts_layout(N, gamma, n_grid, n_bins).total;
  return DSPARK_OK;
}

dspark_status dspark_sts_fit(const dspark_sts_fit_args* a, void* workspace, size_t workspace_bytes, void* stream) {
  if (!a || !sts_dims_ok(a->N, a->gamma, a->n_grid, a->n_bins)) return DSPARK_INVALID_ARG;
  if ((a->N > 0 && (!a->conf_logit || !a->accept_len)) || !a->grid || !a->sts_temp || !a->ece)
    return DSPARK_INVALID_ARG;
  if (!workspace || ((uintptr_t)workspace & 255u)) return DSPARK_INVALID_ARG;
  const StsLayout L = sts_layout(a->N, a->gamma, a->n_grid, a->n_bins);
  if (workspace_bytes < L.total) return DSPARK_INVALID_ARG;
  return cuda_status(launch_sts_fit(*a, static_cast<uint8_t*>(workspace), L, (cudaStream_t)stream));
}

static bool dtype_ok(int32_t dt) { return dt == DSPARK_BF16 || dt == DSPARK_F32; }

// a workspace of at least `need` bytes
static bool ws_ok(const void* ws, size_t bytes, size_t need) {
  return ws && ((uintptr_t)ws & 255u) == 0 && bytes >= need;
}

// rows of `cols` elements `ld` apart whose last element's offset fits 63 bits in bytes
static bool rows_ok(int64_t rows, int64_t cols, int64_t ld) {
  if (rows <= 1) return true;
  return ld >= cols && ld <= (int64_t)1 << 40 && rows <= ((int64_t)1 << 60) / (4 * ld);
}

static bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

dspark_status dspark_quant_fp8(const dspark_quant_fp8_args* a, void* stream) {
  if (!a || a->M < 0 || a->K < 1 || !dtype_ok(a->dtype) || (a->block_rows != 1 && a->block_rows != DSPARK_FP8_BLOCK))
    return DSPARK_INVALID_ARG;
  if (a->M == 0) return DSPARK_OK;
  if (!a->x || !a->codes || !a->scale || !rows_ok(a->M, a->K, a->ldx) || !rows_ok(a->M, a->K, a->ldq))
    return DSPARK_INVALID_ARG;
  if (!aligned_to(a->x, elem_size(a->dtype)) || !aligned_to(a->scale, 4)) return DSPARK_INVALID_ARG;
  if (a->M > kMaxVocabDim || a->K > kMaxVocabDim) return DSPARK_UNSUPPORTED;
  return launched([&] { return launch_quant_fp8(*a, (cudaStream_t)stream); });
}

dspark_status dspark_matmul_fp8_workspace_size(int32_t M, int32_t N, int32_t K, size_t* bytes) {
  if (!bytes || M < 0 || N < 0 || K < 1) return DSPARK_INVALID_ARG;
  if (M > kMaxVocabDim || N > kMaxVocabDim || K > kMaxVocabDim) return DSPARK_UNSUPPORTED;
  *bytes = align_up(matmul_fp8_ws(M, N, K), 256);
  return DSPARK_OK;
}

dspark_status dspark_matmul_fp8(const dspark_matmul_fp8_args* a, void* workspace, size_t workspace_bytes,
                                void* stream) {
  if (!a || a->M < 0 || a->N < 0 || a->K < 1 || !dtype_ok(a->out_dtype)) return DSPARK_INVALID_ARG;
  if (a->M == 0 || a->N == 0) return DSPARK_OK;
  if (!a->a || !a->a_scale || !a->w || !a->w_scale || !a->out) return DSPARK_INVALID_ARG;
  if (!rows_ok(a->M, a->K, a->lda) || !rows_ok(a->N, a->K, a->ldw) || !rows_ok(a->M, a->N, a->ldo))
    return DSPARK_INVALID_ARG;
  if (!aligned16(a->a) || !aligned16(a->w) || (a->M > 1 && a->lda % 16) || (a->N > 1 && a->ldw % 16))
    return DSPARK_INVALID_ARG;
  if (!aligned_to(a->out, elem_size(a->out_dtype)) || !aligned_to(a->a_scale, 4) || !aligned_to(a->w_scale, 4))
    return DSPARK_INVALID_ARG;
  if (!ws_ok(workspace, workspace_bytes, matmul_fp8_ws(a->M, a->N, a->K))) return DSPARK_INVALID_ARG;
  if (a->M > kMaxVocabDim || a->N > kMaxVocabDim || a->K > kMaxVocabDim) return DSPARK_UNSUPPORTED;
  return launched([&] { return launch_matmul_fp8(*a, static_cast<uint8_t*>(workspace), (cudaStream_t)stream); });
}

static dspark_status check_logit_rows(const dspark_logit_rows& r) {
  if (r.N < 0 || r.V < 1 || r.V > DSPARK_MAX_VOCAB || !dtype_ok(r.dtype)) return DSPARK_INVALID_ARG;
  if (r.N == 0) return DSPARK_OK;
  if (!r.logits || !r.tokens || !rows_ok(r.N, r.V, r.ld) || !aligned_to(r.logits, elem_size(r.dtype)))
    return DSPARK_INVALID_ARG;
  if ((r.mark_req != nullptr) != (r.mark_pos != nullptr)) return DSPARK_INVALID_ARG;
  if (r.mark_req && (r.n_req < 0 || r.tok_cols < 0)) return DSPARK_INVALID_ARG;
  if (r.mask && (!aligned_to(r.mask, 4) || !rows_ok(r.N, ((int64_t)r.V + 31) / 32, r.mask_ld)))
    return DSPARK_INVALID_ARG;
  if (r.N > kMaxVocabDim) return DSPARK_UNSUPPORTED;
  return DSPARK_OK;
}

dspark_status dspark_token_logprobs_workspace_size(int32_t N, int32_t V, int32_t top, size_t* bytes) {
  if (!bytes || N < 0 || V < 1 || V > DSPARK_MAX_VOCAB || top < 0) return DSPARK_INVALID_ARG;
  if (top > DSPARK_MAX_TOP || N > kMaxVocabDim) return DSPARK_UNSUPPORTED;
  *bytes = align_up(token_logprobs_ws(N, V, top), 256);
  return DSPARK_OK;
}

dspark_status dspark_token_logprobs(const dspark_token_logprobs_args* a, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  if (!a || a->top < 0) return DSPARK_INVALID_ARG;
  if (a->top > DSPARK_MAX_TOP) return DSPARK_UNSUPPORTED;
  const dspark_status st = check_logit_rows(a->rows);
  if (st != DSPARK_OK || a->rows.N == 0) return st;
  if (a->top > 0 && (!a->top_id || !a->top_logprob)) return DSPARK_INVALID_ARG;
  if (!ws_ok(workspace, workspace_bytes, token_logprobs_ws(a->rows.N, a->rows.V, a->top))) return DSPARK_INVALID_ARG;
  return launched([&] { return launch_token_logprobs(*a, static_cast<uint8_t*>(workspace), (cudaStream_t)stream); });
}

dspark_status dspark_token_logprobs_grad(const dspark_token_logprobs_grad_args* a, void* workspace, void* stream) {
  if (!a || a->top < 0) return DSPARK_INVALID_ARG;
  if (a->top > DSPARK_MAX_TOP) return DSPARK_UNSUPPORTED;
  const dspark_status st = check_logit_rows(a->rows);
  if (st != DSPARK_OK || a->rows.N == 0) return st;
  if (!a->row_stat || !a->grad || (a->g_entropy && !a->entropy) || (a->top > 0 && (!a->top_id || !a->g_top)))
    return DSPARK_INVALID_ARG;
  if (!rows_ok(a->rows.N, a->rows.V, a->ldg) || !aligned_to(a->grad, elem_size(a->rows.dtype)))
    return DSPARK_INVALID_ARG;
  if (a->grad == a->rows.logits && a->rows.N > 1 && a->ldg != a->rows.ld) return DSPARK_INVALID_ARG;
  if (workspace && ((uintptr_t)workspace & 255u)) return DSPARK_INVALID_ARG;
  return launched([&] { return launch_token_logprobs_grad(*a, static_cast<uint8_t*>(workspace), (cudaStream_t)stream); });
}

// The cache's own checks.  kMaxVocabDim keeps rows of the pool and positions in 32 bits.
static dspark_status check_cache(const dspark_kv_cache& c) {
  if (c.n_pages < 1 || c.n_kv_heads < 1 || c.n_req < 0 || c.max_pages < 1) return DSPARK_INVALID_ARG;
  if (c.page_size < 1 || (c.page_size & (c.page_size - 1))) return DSPARK_INVALID_ARG;
  if (c.dtype != DSPARK_E4M3 && c.dtype != DSPARK_BF16) return DSPARK_INVALID_ARG;
  if (c.head_dim < 1) return DSPARK_INVALID_ARG;
  if (c.page_size < 16 || c.page_size > 1024 || (c.head_dim != 64 && c.head_dim != 128)) return DSPARK_UNSUPPORTED;
  if (c.n_pages > kMaxVocabDim / c.page_size || c.n_kv_heads > kMaxVocabDim / c.page_size / c.n_pages ||
      c.max_pages > kMaxVocabDim / c.page_size || c.n_req > kMaxVocabDim)
    return DSPARK_UNSUPPORTED;
  if (!c.k || !c.v || !aligned16(c.k) || !aligned16(c.v)) return DSPARK_INVALID_ARG;
  if (c.dtype == DSPARK_E4M3 && (!c.k_scale || !c.v_scale || !aligned16(c.k_scale) || !aligned16(c.v_scale)))
    return DSPARK_INVALID_ARG;
  if (c.n_req > 0 && (!c.table || !aligned_to(c.table, 4) || !rows_ok(c.n_req, c.max_pages, c.table_ld)))
    return DSPARK_INVALID_ARG;
  return DSPARK_OK;
}

// rows of `cols` elements of `size` bytes for 16-byte accesses
static bool vector_rows_ok(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t size) {
  return p && aligned16(p) && rows_ok(rows, cols, ld) && (rows <= 1 || (ld * size) % 16 == 0);
}

static dspark_status check_cache_rows(const dspark_kv_cache& c, int32_t N, int32_t dtype, const void* k, int64_t ldk,
                                      const void* v, int64_t ldv, const int32_t* mark_req, const int32_t* mark_pos,
                                      const int32_t* base, const int32_t* n_rows, const void* ws) {
  if (N < 0 || !dtype_ok(dtype)) return DSPARK_INVALID_ARG;
  const dspark_status st = check_cache(c);
  if (st != DSPARK_OK || N == 0) return st;
  const int64_t cols = (int64_t)c.n_kv_heads * c.head_dim, size = (int64_t)elem_size(dtype);
  if (!vector_rows_ok(k, N, cols, ldk, size) || !vector_rows_ok(v, N, cols, ldv, size)) return DSPARK_INVALID_ARG;
  if (!mark_req || !mark_pos || (ws && ((uintptr_t)ws & 255u))) return DSPARK_INVALID_ARG;
  for (const void* p : {(const void*)mark_req, (const void*)mark_pos, (const void*)base, (const void*)n_rows})
    if (!aligned_to(p, 4)) return DSPARK_INVALID_ARG;
  if (N > kMaxVocabDim) return DSPARK_UNSUPPORTED;
  return DSPARK_OK;
}

dspark_status dspark_cache_write(const dspark_cache_write_args* a, void* workspace, void* stream) {
  if (!a) return DSPARK_INVALID_ARG;
  const dspark_status st =
      check_cache_rows(a->cache, a->N, a->dtype, a->k, a->ldk, a->v, a->ldv, a->mark_req, a->mark_pos, a->base, a->n_rows,
                       workspace);
  if (st != DSPARK_OK || a->N == 0) return st;
  return launched([&] { return launch_cache_write(*a, static_cast<WsHeader*>(workspace), (cudaStream_t)stream); });
}

dspark_status dspark_cache_read(const dspark_cache_read_args* a, void* workspace, void* stream) {
  if (!a) return DSPARK_INVALID_ARG;
  const dspark_status st =
      check_cache_rows(a->cache, a->N, a->dtype, a->k, a->ldk, a->v, a->ldv, a->mark_req, a->mark_pos, a->base, a->n_rows,
                       workspace);
  if (st != DSPARK_OK || a->N == 0) return st;
  return launched([&] { return launch_cache_read(*a, static_cast<WsHeader*>(workspace), (cudaStream_t)stream); });
}

dspark_status dspark_cache_move(const dspark_cache_move_args* a, void* workspace, void* stream) {
  if (!a || a->path_cols < 1) return DSPARK_INVALID_ARG;
  if (a->path_cols > DSPARK_MAX_TREE) return DSPARK_UNSUPPORTED;
  const dspark_status st = check_cache(a->cache);
  if (st != DSPARK_OK || a->cache.n_req == 0) return st;
  if (!a->base || !a->path || !a->n_path || !rows_ok(a->cache.n_req, a->path_cols, a->path_ld)) return DSPARK_INVALID_ARG;
  if (!aligned_to(a->base, 4) || !aligned_to(a->path, 4) || !aligned_to(a->n_path, 4)) return DSPARK_INVALID_ARG;
  if (workspace && ((uintptr_t)workspace & 255u)) return DSPARK_INVALID_ARG;
  return launched([&] { return launch_cache_move(*a, static_cast<WsHeader*>(workspace), (cudaStream_t)stream); });
}

static dspark_status check_tree_sizes(int32_t n_req, int32_t max_tree, int32_t n_q_heads, int32_t n_kv_heads,
                                      int32_t head_dim) {
  if (n_req < 0 || max_tree < 1 || n_q_heads < 1 || n_kv_heads < 1 || n_q_heads % n_kv_heads || head_dim < 1)
    return DSPARK_INVALID_ARG;
  if (max_tree > DSPARK_MAX_TREE || n_q_heads > (1 << 16) || n_q_heads / n_kv_heads > kMaxTreeGroup || n_req > kMaxVocabDim ||
      (head_dim != 64 && head_dim != 128))
    return DSPARK_UNSUPPORTED;
  return DSPARK_OK;
}

dspark_status dspark_tree_attention_workspace_size(int32_t n_req, int32_t max_tree, int32_t n_q_heads, int32_t n_kv_heads,
                                                   int32_t head_dim, size_t* bytes) {
  if (!bytes) return DSPARK_INVALID_ARG;
  const dspark_status st = check_tree_sizes(n_req, max_tree, n_q_heads, n_kv_heads, head_dim);
  if (st == DSPARK_OK) *bytes = align_up(tree_attention_ws(max_tree, n_q_heads, n_kv_heads, head_dim), 256);
  return st;
}

dspark_status dspark_tree_attention(const dspark_tree_attention_args* a, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  if (!a || a->N < 0 || !isfinite(a->scale)) return DSPARK_INVALID_ARG;
  const dspark_kv_cache& c = a->cache;
  dspark_status st = check_cache(c);
  if (st != DSPARK_OK) return st;
  st = check_tree_sizes(c.n_req, a->max_tree, a->n_q_heads, c.n_kv_heads, c.head_dim);
  if (st != DSPARK_OK || a->N == 0 || c.n_req == 0) return st;
  const int64_t cols = (int64_t)a->n_q_heads * c.head_dim;
  if (!vector_rows_ok(a->q, a->N, cols, a->ldq, 2) || !vector_rows_ok(a->out, a->N, cols, a->ldo, 2))
    return DSPARK_INVALID_ARG;
  if (!a->offsets || !a->base || !aligned_to(a->offsets, 4) || !aligned_to(a->base, 4) || !aligned_to(a->tree, 8))
    return DSPARK_INVALID_ARG;
  if (!ws_ok(workspace, workspace_bytes, tree_attention_ws(a->max_tree, a->n_q_heads, c.n_kv_heads, c.head_dim)))
    return DSPARK_INVALID_ARG;
  if (a->N > kMaxVocabDim) return DSPARK_UNSUPPORTED;
  return launched([&] { return launch_tree_attention(*a, static_cast<uint8_t*>(workspace), (cudaStream_t)stream); });
}

}  // extern "C"
