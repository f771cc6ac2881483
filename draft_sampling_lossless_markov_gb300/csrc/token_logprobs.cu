// Log probability and rank of a given token, entropy and top alternatives of
// rows of logits, and their gradient.  With c = log2(e) / T, m a row's largest
// candidate and t = (logit - m) c:
//     S = sum 2^t, A = sum t 2^t, ln p = (logit - m) / T - ln S,
//     entropy = ln S - ln 2 A / S,
//     d(v) = (1 / T) (picked(v) - p(v) (G + g_H (ln p(v) + entropy))).
//
// Both kernels read a row once in 16-byte vectors (the gradient also writes it
// once) and are bounded by memory as long as the arithmetic stays below some
// ten instructions an element; hence packed fp32 pairs and the approximate
// base-2 exponential (2 ulp), with fp32 sums.  A cluster of CTAs splits a row
// when there are few rows; the parts meet in distributed shared memory in rank
// order (no atomics on results: equal calls give equal bits).
//
// t is clamped to [-200, ..]: 2^t is 0 there, and 0 t stays 0 for logits of -inf
// or the type's lowest value.  NaN passes the clamp and makes S NaN.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace dspark {

namespace {

constexpr int LT = 256;  // threads
constexpr int LW = LT / 32;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.402823466e+38f;
constexpr int kMaxSplit = 8;

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------
struct RowMeta {
  int tok;  // -1: none
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

__device__ __forceinline__ float shifted(float a, float m, float c) { return ptx::max_nan((a - m) * c, -200.f); }

__device__ __forceinline__ bool mask_bit(const uint32_t* mask, int v) {
  return !mask || ((mask[v >> 5] >> (v & 31)) & 1u);
}
// bits v .. v + 7 (all inside the vocabulary)
__device__ __forceinline__ uint32_t mask8(const uint32_t* mask, int v) {
  const int w = v >> 5, o = v & 31;
  uint32_t b = mask[w] >> o;
  if (o > 24) b |= mask[w + 1] << (32 - o);
  return b & 255u;
}

// A row as vectors of 8 elements from its first 16-byte boundary on: elements
// head .. head + 8 nv - 1; the up to 14 others are `edge` elements.
struct RowShape {
  int head, nv, V;
  __device__ __forceinline__ int n_edge() const { return V - 8 * nv; }
  __device__ __forceinline__ int edge(int j) const { return j < head ? j : j + 8 * nv; }
};
template <typename T>
__device__ __forceinline__ RowShape row_shape(const T* row, int V) {
  RowShape s;
  s.V = V;
  s.head = min(V, (int)(((16u - ((uint32_t)(uintptr_t)row & 15u)) & 15u) / sizeof(T)));
  s.nv = (V - s.head) / 8;
  return s;
}

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// eight elements as loaded
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void fill_neg_inf() { a = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&d)[8], bool vec) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(d[2 * i], d[2 * i + 1]);
    if (vec) {
      __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(h));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[2 * i] = h[i].x;
        p[2 * i + 1] = h[i].y;
      }
    }
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void fill_neg_inf() { a = b = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&d)[8], bool vec) {
    if (vec) {
      __stcs(reinterpret_cast<float4*>(p), make_float4(d[0], d[1], d[2], d[3]));
      __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(d[4], d[5], d[6], d[7]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = d[i];
    }
  }
};

// ---------------------------------------------------------------------------
// log probabilities
// ---------------------------------------------------------------------------
// m, S, A of some elements; m is kLowest and S 0 where there is no candidate
struct Stat {
  float m, S, A;
};
__device__ __forceinline__ void stat_merge(Stat& a, const Stat& b, float c) {
  const float m = fmaxf(a.m, b.m);
  const float da = shifted(a.m, m, c), db = shifted(b.m, m, c);
  const float fa = ptx::ex2(da), fb = ptx::ex2(db);
  a.A = fa * (a.A + da * a.S) + fb * (b.A + db * b.S);
  a.S = fa * a.S + fb * b.S;
  a.m = m;
}

// (logit, id) as one number, larger for what comes first in the order (logit
// descending, id ascending); + 0 makes -0 equal to 0; 0 is below every candidate
__device__ __forceinline__ uint64_t order_key(float x, int v) {
  uint32_t b = __float_as_uint(x + 0.f);
  b = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((uint64_t)b << 32) | (uint32_t)(0x7FFFFFFF - v);
}
__device__ __forceinline__ float key_logit(uint64_t k) {
  const uint32_t b = (uint32_t)(k >> 32);
  return __uint_as_float((b & 0x80000000u) ? (b & 0x7FFFFFFFu) : ~b);
}
__device__ __forceinline__ int key_id(uint64_t k) { return 0x7FFFFFFF - (int)(uint32_t)k; }

// the largest float below x (finite or +inf)
__device__ __forceinline__ float float_below(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return __uint_as_float((b & 0x80000000u) ? b + 1 : b == 0 ? 0x80000001u : b - 1);
}

__device__ __forceinline__ uint64_t warp_desc_merge(uint64_t k, int lane) {  // bitonic sequence to descending
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t other = __shfl_xor_sync(0xffffffffu, k, o);
    k = ((lane & o) == 0) == (k > other) ? k : other;
  }
  return k;
}
__device__ __forceinline__ uint64_t warp_desc_sort(uint64_t k, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int o = size >> 1; o > 0; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(0xffffffffu, k, o);
      const bool first = (lane & o) == 0, desc = (lane & size) == 0;
      k = (first == desc) == (k > other) ? k : other;
    }
  return k;
}
// the 32 largest of a descending list and a batch (one number a lane each), descending
__device__ __forceinline__ uint64_t warp_top_merge(uint64_t list, uint64_t batch, int lane) {
  batch = warp_desc_sort(batch, lane);
  const uint64_t rev = __shfl_sync(0xffffffffu, batch, 31 - lane);
  return warp_desc_merge(list > rev ? list : rev, lane);
}

constexpr int kCap = 2048;  // candidate buffer: one vector a thread always fits

struct LpShared {
  Stat st[LW];
  int cnt[LW];
  float jth[LW];
  // the CTA's results, read by rank 0 of the cluster
  Stat part;
  int part_cnt;
  uint64_t list[32];
};
struct TopShared {
  uint64_t thr;   // the K-th best key so far: later keys must be larger
  int n;          // candidates in the buffer
  uint64_t buf[kCap];
};

// CTA state of the top-K search; every function is called by all threads
template <bool kTop>
struct TopSearch {
  TopShared* s;
  uint64_t list;  // warp 0: the best 32 so far, one a lane, descending
  int k;
  __device__ __forceinline__ void append(float x, int v, uint64_t thr) {
    const uint64_t key = order_key(x, v);
    if (x > -INFINITY && key > thr) {
      const int at = atomicAdd(&s->n, 1);
      if (at < kCap) s->buf[at] = key;
    }
  }
  // take the buffer into the list and raise the threshold (after a barrier; ends with one)
  __device__ __forceinline__ void absorb() {
    const int lane = threadIdx.x & 31;
    const int n = s->n;
    if (n > 0) {
      __syncthreads();  // everybody has read n
      if (threadIdx.x < 32) {
        for (int b = 0; b < n; b += 32) {
          const uint64_t key = b + lane < n ? s->buf[b + lane] : 0;
          const uint64_t last = __shfl_sync(0xffffffffu, list, k - 1);
          if (__any_sync(0xffffffffu, key > last)) list = warp_top_merge(list, key, lane);
        }
        const uint64_t last = __shfl_sync(0xffffffffu, list, k - 1);
        if (lane == 0) {
          s->thr = last > s->thr ? last : s->thr;
          s->n = 0;
        }
      }
    }
    __syncthreads();
  }
};

template <typename T, bool kTop>
__global__ void __launch_bounds__(LT, 4) k_logprobs(const dspark_token_logprobs_args p, WsHeader* hdr, int split) {
  constexpr int U = std::is_same<T, float>::value ? 2 : 4;  // vectors of a thread and chunk
  const dspark_logit_rows& r = p.rows;
  const int i = blockIdx.x / split, rank = blockIdx.x % split;
  if (r.n_rows && i >= *r.n_rows) return;  // the whole cluster
  __shared__ LpShared sh;
  extern __shared__ __align__(16) uint8_t dyn[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const RowMeta meta = row_meta(r, i, hdr, tid == 0 && rank == 0);
  const T* row = static_cast<const T*>(r.logits) + (int64_t)i * r.ld;
  const uint32_t* mask = r.mask ? r.mask + (int64_t)i * r.mask_ld : nullptr;
  const float c = log2_scale(meta.T);
  const RowShape shp = row_shape(row, r.V);
  const int v0 = (int)((int64_t)shp.nv * rank / split), v1 = (int)((int64_t)shp.nv * (rank + 1) / split);
  const T* base = row + shp.head;

  // rank: x > x_hi counts from the token's vector on, x > x_lo (x >= x_token) before it
  const bool given = meta.tok >= 0 && mask_bit(mask, meta.tok);
  const float xt = given ? to_f32(row[meta.tok]) : -INFINITY;
  const bool has = given && !(xt == -INFINITY);
  const float x_hi = has ? xt : INFINITY, x_lo = has ? float_below(xt) : INFINITY;
  const int tok_vec = has ? (meta.tok < shp.head ? -1 : (meta.tok - shp.head) / 8) : -1;

  TopSearch<kTop> top{reinterpret_cast<TopShared*>(dyn), 0, p.top};
  if (kTop && tid == 0) {
    top.s->thr = 0;
    top.s->n = 0;
  }

  float m = kLowest;
  uint64_t S2 = 0, A2 = 0;
  const uint64_t c2 = ptx::pack2(c, c);
  int ahead = 0;

  const auto masked = [&](float(&x)[8], int j) {
    if (mask) {
      const uint32_t b = mask8(mask, shp.head + 8 * j);
      if (b != 255u) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!((b >> e) & 1u)) x[e] = -INFINITY;
      }
    }
  };
  const auto max8 = [](const float(&x)[8]) {
    return fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
  };
  // sums and rank of vector j; returns its largest element
  const auto add = [&](float(&x)[8], int j) {
    masked(x, j);
    const float cm = max8(x);
    if (cm > m) {
      const float d = shifted(m, cm, c), f = ptx::ex2(d);
      const uint64_t d2 = ptx::pack2(d, d), f2 = ptx::pack2(f, f);
      A2 = ptx::mul2(f2, ptx::fma2(d2, S2, A2));
      S2 = ptx::mul2(f2, S2);
      m = cm;
    }
    const uint64_t nm = ptx::pack2(-m, -m);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float2 t = ptx::unpack2(ptx::mul2(ptx::add2(ptx::pack2(x[e], x[e + 1]), nm), c2));
      const float t0 = ptx::max_nan(t.x, -200.f), t1 = ptx::max_nan(t.y, -200.f);
      const uint64_t e2 = ptx::pack2(ptx::ex2(t0), ptx::ex2(t1));
      S2 = ptx::add2(S2, e2);
      A2 = ptx::fma2(e2, ptx::pack2(t0, t1), A2);
    }
    const float xr = j < tok_vec ? x_lo : x_hi;
#pragma unroll
    for (int e = 0; e < 8; ++e) ahead += x[e] > xr;
    if (j == tok_vec) {
#pragma unroll
      for (int e = 0; e < 8; ++e) ahead += x[e] == xt && shp.head + 8 * j + e < meta.tok;
    }
    return cm;
  };
  const auto offer = [&](const float(&x)[8], int j, uint64_t thr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) top.append(x[e], shp.head + 8 * j + e, thr);
  };

  if (kTop) __syncthreads();
  bool first = true;
  for (int j0 = v0; j0 < v1; j0 += U * LT) {
    Vec8<T> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * LT + tid;
      if (j < v1)
        raw[u].load(base + 8 * (int64_t)j);
      else
        raw[u].fill_neg_inf();
    }
    uint64_t thr = 0;
    float thr_x = -INFINITY;
    if (kTop && !first) {
      thr = top.s->thr;
      thr_x = thr ? key_logit(thr) : -INFINITY;
    }
    float cm[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * LT + tid;
      float x[8];
      raw[u].get(x);
      cm[u] = -INFINITY;
      if (j < v1) cm[u] = add(x, j);
      if (kTop && !first && j < v1 && cm[u] >= thr_x) offer(x, j, thr);
    }
    if (kTop) {
      if (first) {
        // a first threshold: LW j-th largest thread maxima are at least K elements
        first = false;
        float mine = cm[0];
#pragma unroll
        for (int u = 1; u < U; ++u) mine = fmaxf(mine, cm[u]);
        float jth = -INFINITY;
        for (int n = (p.top + LW - 1) / LW; n > 0; --n) {
          jth = warp_max(mine);
          const unsigned at = __ballot_sync(0xffffffffu, mine == jth);
          if (lane == __ffs(at) - 1) mine = -INFINITY;
        }
        if (lane == 0) sh.jth[warp] = jth;
        __syncthreads();
        float lo = sh.jth[0];
#pragma unroll
        for (int w = 1; w < LW; ++w) lo = fminf(lo, sh.jth[w]);
        // the key below every key of that logit
        thr = lo > -INFINITY ? order_key(lo, 0x7FFFFFFF) : 0;
        thr_x = lo;
        if (tid == 0) top.s->thr = thr;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = j0 + u * LT + tid;
          if (j < v1 && cm[u] >= thr_x) {
            float x[8];
            raw[u].get(x);
            masked(x, j);
            offer(x, j, thr);
          }
        }
      }
      __syncthreads();
      if (top.s->n <= kCap) {
        top.absorb();
      } else {
        // more than the buffer holds: the chunk again, a vector a thread at a time
        __syncthreads();
        if (tid == 0) top.s->n = 0;
        __syncthreads();
#pragma unroll 1
        for (int u = 0; u < U; ++u) {
          const int j = j0 + u * LT + tid;
          thr = top.s->thr;
          float x[8];
          bool in = false;
#pragma unroll
          for (int w = 0; w < U; ++w)
            if (w == u) {
              raw[w].get(x);
              in = j < v1 && cm[w] >= (thr ? key_logit(thr) : -INFINITY);
            }
          if (in) {
            masked(x, j);
            offer(x, j, thr);
          }
          __syncthreads();
          top.absorb();
        }
      }
    }
  }
  // the elements outside the vectors, one a thread
  if (rank == 0) {
    if (tid < shp.n_edge()) {
      const int v = shp.edge(tid);
      float x = to_f32(row[v]);
      if (!mask_bit(mask, v)) x = -INFINITY;
      if (x > m) {
        const float d = shifted(m, x, c), f = ptx::ex2(d);
        const uint64_t d2 = ptx::pack2(d, d), f2 = ptx::pack2(f, f);
        A2 = ptx::mul2(f2, ptx::fma2(d2, S2, A2));
        S2 = ptx::mul2(f2, S2);
        m = x;
      }
      const float t = shifted(x, m, c), e = ptx::ex2(t);
      S2 = ptx::add2(S2, ptx::pack2(e, 0.f));
      A2 = ptx::add2(A2, ptx::pack2(e * t, 0.f));
      ahead += x > x_hi || (x == xt && v < meta.tok);
      if (kTop) top.append(x, v, top.s->thr);
    }
    if (kTop) {
      __syncthreads();
      top.absorb();
    }
  }

  // warp, CTA, cluster
  const float2 Sp = ptx::unpack2(S2), Ap = ptx::unpack2(A2);
  Stat st{m, Sp.x + Sp.y, Ap.x + Ap.y};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Stat b{__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.S, o),
                 __shfl_xor_sync(0xffffffffu, st.A, o)};
    stat_merge(st, b, c);
    ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
  }
  if (lane == 0) {
    sh.st[warp] = st;
    sh.cnt[warp] = ahead;
  }
  __syncthreads();
  if (warp == 0) {
    st = sh.st[0];
    ahead = sh.cnt[0];
#pragma unroll
    for (int w = 1; w < LW; ++w) {
      stat_merge(st, sh.st[w], c);
      ahead += sh.cnt[w];
    }
  }
  if (split > 1) {
    if (warp == 0) {
      if (lane == 0) {
        sh.part = st;
        sh.part_cnt = ahead;
      }
      if (kTop) sh.list[lane] = top.list;
      __syncwarp();
    }
    ptx::cluster_sync();
    if (warp == 0 && rank == 0) {
      for (int q = 1; q < split; ++q) {
        const Stat b{ptx::ld_cluster_f32(ptx::map_to_rank(&sh.part.m, q)), ptx::ld_cluster_f32(ptx::map_to_rank(&sh.part.S, q)),
                     ptx::ld_cluster_f32(ptx::map_to_rank(&sh.part.A, q))};
        stat_merge(st, b, c);
        ahead += __float_as_int(ptx::ld_cluster_f32(ptx::map_to_rank(&sh.part_cnt, q)));
        if (kTop) {
          const uint64_t b64 = ptx::ld_cluster_u64(ptx::map_to_rank(&sh.list[lane], q));
          const uint64_t rev = __shfl_sync(0xffffffffu, b64, 31 - lane);
          top.list = warp_desc_merge(top.list > rev ? top.list : rev, lane);
        }
      }
    }
    ptx::cluster_sync();
  }
  if (warp == 0 && rank == 0) {
    const bool empty = st.S == 0.f, bad = isnan(st.S);
    const float logS = logf(st.S);
    if (lane == 0) {
      if (p.logprob)
        p.logprob[i] = meta.tok < 0 ? 0.f : bad ? NAN : !has ? -INFINITY : __fdiv_rn(xt - st.m, meta.T) - logS;
      if (p.entropy) p.entropy[i] = empty ? 0.f : bad ? NAN : logS - __fdiv_rn(st.A, st.S) * kLn2;
      if (p.rank) p.rank[i] = has && !bad ? ahead : -1;
      if (p.row_stat) {
        p.row_stat[2 * (int64_t)i] = empty ? -INFINITY : st.m;
        p.row_stat[2 * (int64_t)i + 1] = st.S;
      }
    }
    if (kTop && lane < p.top) {
      const bool found = top.list != 0 && !bad;
      p.top_id[(int64_t)i * p.top + lane] = found ? key_id(top.list) : -1;
      p.top_logprob[(int64_t)i * p.top + lane] =
          bad ? NAN : found ? __fdiv_rn(key_logit(top.list) - st.m, meta.T) - logS : -INFINITY;
    }
  }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(LT, 4) k_logprobs_grad(const dspark_token_logprobs_grad_args p, WsHeader* hdr,
                                                         int split) {
  constexpr int U = std::is_same<T, float>::value ? 2 : 4;
  const dspark_logit_rows& r = p.rows;
  const int i = blockIdx.x / split, rank = blockIdx.x % split;
  if (r.n_rows && i >= *r.n_rows) return;  // the whole cluster
  __shared__ int pid[DSPARK_MAX_TOP + 1];
  __shared__ float pg[DSPARK_MAX_TOP + 1], px[DSPARK_MAX_TOP + 1];
  const int tid = threadIdx.x;
  const RowMeta meta = row_meta(r, i, hdr, tid == 0 && rank == 0);
  const T* row = static_cast<const T*>(r.logits) + (int64_t)i * r.ld;
  T* out = static_cast<T*>(p.grad) + (int64_t)i * p.ldg;
  const uint32_t* mask = r.mask ? r.mask + (int64_t)i * r.mask_ld : nullptr;
  const RowShape shp = row_shape(row, r.V);
  const int v0 = (int)((int64_t)shp.nv * rank / split), v1 = (int)((int64_t)shp.nv * (rank + 1) / split);
  // the picked places: the token, then the alternatives; -1 where the term is left out
  const int np = p.top + 1;
  if (tid < np) {
    int id = tid == 0 ? (p.g_logprob ? meta.tok : -1) : p.top_id[(int64_t)i * p.top + tid - 1];
    float x = -INFINITY;
    if (id >= 0 && id < r.V && mask_bit(mask, id)) x = to_f32(row[id]);
    if (x == -INFINITY) id = -1;
    pid[tid] = id;
    px[tid] = x;
    pg[tid] = id < 0 ? 0.f : tid == 0 ? p.g_logprob[i] : p.g_top[(int64_t)i * p.top + tid - 1];
  }
  __syncthreads();
  // the gradient may replace the logits: every CTA of the row has read its picks
  if (split > 1) ptx::cluster_sync();
  const float c = log2_scale(meta.T);
  const float m = p.row_stat[2 * (int64_t)i], S = p.row_stat[2 * (int64_t)i + 1];
  const float gH = p.g_entropy ? p.g_entropy[i] : 0.f, H = p.g_entropy ? p.entropy[i] : 0.f;
  float G = 0.f;
  for (int k = 0; k < np; ++k) G += pg[k];
  // d = -p (alpha + beta t) with 1 / T inside
  const float inv_s = __fdiv_rn(1.f, S);
  const float alpha = __fdiv_rn(G + gH * (H - logf(S)), meta.T), beta = __fdiv_rn(gH * kLn2, meta.T);
  const auto grad = [&](float x) {
    const float t = shifted(x, m, c);
    const float d = -(ptx::ex2(t) * inv_s) * fmaf(beta, t, alpha);
    return x == -INFINITY ? 0.f : d;
  };
  const T* base = row + shp.head;
  T* obase = out + shp.head;
  const bool vec = ((uintptr_t)obase & 15u) == 0;
  for (int j0 = v0; j0 < v1; j0 += U * LT) {
    Vec8<T> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * LT + tid;
      if (j < v1) raw[u].load(base + 8 * (int64_t)j);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * LT + tid;
      if (j >= v1) continue;
      float x[8];
      raw[u].get(x);
      if (mask) {
        const uint32_t b = mask8(mask, shp.head + 8 * j);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!((b >> e) & 1u)) x[e] = -INFINITY;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = grad(x[e]);
      Vec8<T>::store(obase + 8 * (int64_t)j, x, vec);
    }
  }
  if (rank == 0 && tid < shp.n_edge()) {
    const int v = shp.edge(tid);
    const float d = grad(mask_bit(mask, v) ? to_f32(row[v]) : -INFINITY);
    out[v] = from_f32<T>(d);
  }
  __syncthreads();
  // the picked places again, with what was picked there (the first of equal ids does it)
  if (tid < np && pid[tid] >= 0) {
    const int v = pid[tid];
    const int j = v < shp.head ? -1 : (v - shp.head) / 8;
    const bool here = j >= 0 && j < shp.nv ? j >= v0 && j < v1 : rank == 0;
    float pick = 0.f;
    bool mine = here;
    for (int k = 0; k < np; ++k)
      if (pid[k] == v) {
        if (k < tid) mine = false;
        pick += pg[k];
      }
    if (mine) out[v] = from_f32<T>(__fdiv_rn(pick, meta.T) + grad(px[tid]));
  }
}

// CTAs a row is split over
int row_split(int64_t N, int64_t V) {
  int split = 1;
  while (split < kMaxSplit && N * split * 2 <= 608 && V >= 4096 * split) split *= 2;
  return split;
}

template <typename K, typename A>
cudaError_t launch_rows(K kernel, const A& a, WsHeader* hdr, int N, int split, unsigned smem, cudaStream_t s) {
  cudaLaunchConfig_t c = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)split;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  c.gridDim = dim3((unsigned)N * (unsigned)split);
  c.blockDim = dim3(LT);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  c.attrs = at;
  c.numAttrs = split > 1 ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&c, kernel, a, hdr, split);
  if (e != cudaSuccess) return e;
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

size_t token_logprobs_ws(int, int, int) { return sizeof(WsHeader); }

cudaError_t launch_token_logprobs(const dspark_token_logprobs_args& a, uint8_t* ws, cudaStream_t s) {
  WsHeader* hdr = reinterpret_cast<WsHeader*>(ws);
  const int N = a.rows.N, split = row_split(N, a.rows.V);
  const bool bf16 = a.rows.dtype == DSPARK_BF16;
  if (a.top > 0)
    return bf16 ? launch_rows(k_logprobs<__nv_bfloat16, true>, a, hdr, N, split, sizeof(TopShared), s)
                : launch_rows(k_logprobs<float, true>, a, hdr, N, split, sizeof(TopShared), s);
  return bf16 ? launch_rows(k_logprobs<__nv_bfloat16, false>, a, hdr, N, split, 0, s)
              : launch_rows(k_logprobs<float, false>, a, hdr, N, split, 0, s);
}

cudaError_t launch_token_logprobs_grad(const dspark_token_logprobs_grad_args& a, uint8_t* ws, cudaStream_t s) {
  WsHeader* hdr = reinterpret_cast<WsHeader*>(ws);
  const int N = a.rows.N, split = row_split(N, a.rows.V);
  return a.rows.dtype == DSPARK_BF16 ? launch_rows(k_logprobs_grad<__nv_bfloat16>, a, hdr, N, split, 0, s)
                                     : launch_rows(k_logprobs_grad<float>, a, hdr, N, split, 0, s);
}

}  // namespace dspark
