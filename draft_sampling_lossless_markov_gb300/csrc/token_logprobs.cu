// Log probability and rank of a given token, entropy and top alternatives of
// rows of logits, and their gradient.  With y = (logit - m) / T over a row's
// candidates, m their largest logit:
//     S = sum e^y, ln p(v) = y_v - ln S, entropy = ln S - (sum y e^y) / S,
//     d(v) = (1/T) (picked(v) - p(v) (G + g_H (ln p(v) + entropy))).
// One pass over the row keeps a running (m, S, sum y e^y) per thread; a larger
// m rescales them.  Bounded by memory: the logits are read once (and the
// gradient written once).
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace dspark {

namespace {

constexpr int LT = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct RowMeta {
  int tok;      // -1: none
  float T;
};

// token and temperature of row i; reports what is outside its range
__device__ __forceinline__ RowMeta row_meta(const dspark_logit_rows& r, int i, WsHeader* hdr, bool report) {
  RowMeta m{-1, 1.f};
  int64_t at = i;
  int ti = i;
  if (r.mark_req) {
    const int q = r.mark_req[i], pos = r.mark_pos[i];
    if (q == -1) return m;
    if (q < 0 || q >= r.n_req || pos < 0 || pos >= r.tok_cols) {
      if (report && hdr) report_error(hdr, DSPARK_BAD_INPUT, i);
      return m;
    }
    at = (int64_t)q * r.tok_cols + pos;
    ti = q;
  }
  const int t = r.tokens[at];
  if (t >= 0 && t < r.V)
    m.tok = t;
  else if (t != -1 && report && hdr)
    report_error(hdr, DSPARK_BAD_INPUT, i);
  if (r.temp) {
    const float T = r.temp[ti];
    if (T > 0.f && T < INFINITY) m.T = T;
  }
  return m;
}

// log2(e) / T, finite for every T > 0 so that 0 * c is 0
__device__ __forceinline__ float log2_scale(float T) { return fminf(__fdiv_rn(kLog2e, T), 3.0e38f); }

__device__ __forceinline__ bool mask_bit(const dspark_logit_rows& r, int i, int v) {
  return !r.mask || ((r.mask[(int64_t)i * r.mask_ld + (v >> 5)] >> (v & 31)) & 1u);
}

// (a - m) c clamped to where 2^x is 0, so that 0 * x stays 0; NaN stays NaN
__device__ __forceinline__ float shifted(float a, float m, float c) {
  const float t = (a - m) * c;
  return t < -200.f ? -200.f : t;
}

struct Stat {
  float m, S, A;  // largest logit, sum 2^t, sum t 2^t with t = (logit - m) c
};

__device__ __forceinline__ void stat_merge(Stat& a, const Stat& b, float c) {
  if (b.m == -INFINITY) return;
  if (a.m == -INFINITY) {
    a = b;
    return;
  }
  const float m = fmaxf(a.m, b.m);
  const float da = shifted(a.m, m, c), db = shifted(b.m, m, c);
  const float fa = exp2f(da), fb = exp2f(db);
  a.A = fa * (a.A + da * a.S) + fb * (b.A + db * b.S);
  a.S = fa * a.S + fb * b.S;
  a.m = m;
}

// (logit, id) as one number that orders by logit descending, id ascending
// (larger first); + 0 makes -0 equal to 0
__device__ __forceinline__ uint64_t order_key(float x, int v) {
  uint32_t b = __float_as_uint(x + 0.f);
  b = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((uint64_t)b << 32) | (uint32_t)(0x7FFFFFFF - v);
}

template <typename T>
__global__ void __launch_bounds__(LT) k_logprobs_simple(const dspark_token_logprobs_args p, WsHeader* hdr) {
  const dspark_logit_rows& r = p.rows;
  const int i = blockIdx.x;
  if (r.n_rows && i >= *r.n_rows) return;
  __shared__ Stat st[LT];
  __shared__ int cnt[LT];
  __shared__ uint64_t best[LT];
  const RowMeta meta = row_meta(r, i, hdr, threadIdx.x == 0);
  const T* row = static_cast<const T*>(r.logits) + (int64_t)i * r.ld;
  const float c = log2_scale(meta.T);
  const bool has = meta.tok >= 0 && mask_bit(r, i, meta.tok) && !(to_f32(row[meta.tok]) == -INFINITY);
  const float xt = has ? to_f32(row[meta.tok]) : 0.f;
  const uint64_t kt = has ? order_key(xt, meta.tok) : 0;
  Stat s{-INFINITY, 0.f, 0.f};
  int ahead = 0;
  for (int v = threadIdx.x; v < r.V; v += LT) {
    if (!mask_bit(r, i, v)) continue;
    const float x = to_f32(row[v]);
    if (x == -INFINITY) continue;
    if (isnan(x)) {
      s.m = fmaxf(s.m, -3e38f);
      s.S = NAN;
      continue;
    }
    stat_merge(s, Stat{x, x == INFINITY ? NAN : 1.f, 0.f}, c);
    if (has) ahead += order_key(x, v) > kt;
  }
  st[threadIdx.x] = s;
  cnt[threadIdx.x] = ahead;
  __syncthreads();
  for (int o = LT / 2; o > 0; o >>= 1) {
    if (threadIdx.x < o) {
      stat_merge(st[threadIdx.x], st[threadIdx.x + o], c);
      cnt[threadIdx.x] += cnt[threadIdx.x + o];
    }
    __syncthreads();
  }
  s = st[0];
  const bool empty = s.m == -INFINITY, bad = isnan(s.S);
  const float logS = logf(s.S);
  if (threadIdx.x == 0) {
    if (p.logprob) p.logprob[i] = meta.tok < 0 ? 0.f : bad ? NAN : !has ? -INFINITY : __fdiv_rn(xt - s.m, meta.T) - logS;
    if (p.entropy) p.entropy[i] = empty ? 0.f : bad ? NAN : logS - __fdiv_rn(s.A, s.S) * kLn2;
    if (p.rank) p.rank[i] = has && !bad ? cnt[0] : -1;
    if (p.row_stat) {
      p.row_stat[2 * (int64_t)i] = s.m;
      p.row_stat[2 * (int64_t)i + 1] = s.S;
    }
  }
  uint64_t below = ~0ull;
  for (int k = 0; k < p.top; ++k) {
    uint64_t b = 0;
    if (!bad)
      for (int v = threadIdx.x; v < r.V; v += LT) {
        if (!mask_bit(r, i, v)) continue;
        const float x = to_f32(row[v]);
        if (x == -INFINITY) continue;
        const uint64_t key = order_key(x, v);
        if (key < below && key > b) b = key;
      }
    best[threadIdx.x] = b;
    __syncthreads();
    for (int o = LT / 2; o > 0; o >>= 1) {
      if (threadIdx.x < o) best[threadIdx.x] = max(best[threadIdx.x], best[threadIdx.x + o]);
      __syncthreads();
    }
    below = best[0];
    __syncthreads();
    if (threadIdx.x == 0) {
      const int id = below ? 0x7FFFFFFF - (int)(uint32_t)below : -1;
      p.top_id[(int64_t)i * p.top + k] = id;
      p.top_logprob[(int64_t)i * p.top + k] =
          bad ? NAN : id < 0 ? -INFINITY : __fdiv_rn(to_f32(row[id]) - s.m, meta.T) - logS;
    }
  }
}

__device__ __forceinline__ void store_grad(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T>
__global__ void __launch_bounds__(LT) k_grad_simple(const dspark_token_logprobs_grad_args p, WsHeader* hdr) {
  const dspark_logit_rows& r = p.rows;
  const int i = blockIdx.x;
  if (r.n_rows && i >= *r.n_rows) return;
  __shared__ int pid[DSPARK_MAX_TOP + 1];
  __shared__ float pg[DSPARK_MAX_TOP + 1];
  const RowMeta meta = row_meta(r, i, hdr, threadIdx.x == 0);
  const T* row = static_cast<const T*>(r.logits) + (int64_t)i * r.ld;
  T* out = static_cast<T*>(p.grad) + (int64_t)i * p.ldg;
  const int np = p.top + 1;
  if (threadIdx.x < np) {
    int id = threadIdx.x == 0 ? (p.g_logprob ? meta.tok : -1) : p.top_id[(int64_t)i * p.top + threadIdx.x - 1];
    if (id < 0 || id >= r.V || !mask_bit(r, i, id) || to_f32(row[id]) == -INFINITY) id = -1;
    pid[threadIdx.x] = id;
    pg[threadIdx.x] = id < 0 ? 0.f : threadIdx.x == 0 ? p.g_logprob[i] : p.g_top[(int64_t)i * p.top + threadIdx.x - 1];
  }
  __syncthreads();
  const float c = log2_scale(meta.T);
  const float m = p.row_stat[2 * (int64_t)i], S = p.row_stat[2 * (int64_t)i + 1];
  const float gH = p.g_entropy ? p.g_entropy[i] : 0.f, H = p.g_entropy ? p.entropy[i] : 0.f;
  float G = 0.f;
  for (int k = 0; k < np; ++k) G += pg[k];
  const float logS = logf(S);
  for (int v = threadIdx.x; v < r.V; v += LT) {
    float d = 0.f;
    if (mask_bit(r, i, v) && m > -INFINITY) {
      const float x = to_f32(row[v]);
      if (x != -INFINITY) {
        const float t = shifted(x, m, c);
        float pick = 0.f;
        for (int k = 0; k < np; ++k)
          if (pid[k] == v) pick += pg[k];
        d = __fdiv_rn(pick - __fdiv_rn(exp2f(t), S) * (G + gH * (t * kLn2 - logS + H)), meta.T);
      }
    }
    store_grad(out + v, d);
  }
}

}  // namespace

size_t token_logprobs_ws(int, int, int) { return sizeof(WsHeader); }

cudaError_t launch_token_logprobs(const dspark_token_logprobs_args& a, uint8_t* ws, cudaStream_t s) {
  WsHeader* hdr = reinterpret_cast<WsHeader*>(ws);
  if (a.rows.dtype == DSPARK_BF16)
    k_logprobs_simple<__nv_bfloat16><<<a.rows.N, LT, 0, s>>>(a, hdr);
  else
    k_logprobs_simple<float><<<a.rows.N, LT, 0, s>>>(a, hdr);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_token_logprobs_grad(const dspark_token_logprobs_grad_args& a, uint8_t* ws, cudaStream_t s) {
  WsHeader* hdr = reinterpret_cast<WsHeader*>(ws);
  if (a.rows.dtype == DSPARK_BF16)
    k_grad_simple<__nv_bfloat16><<<a.rows.N, LT, 0, s>>>(a, hdr);
  else
    k_grad_simple<float><<<a.rows.N, LT, 0, s>>>(a, hdr);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace dspark
