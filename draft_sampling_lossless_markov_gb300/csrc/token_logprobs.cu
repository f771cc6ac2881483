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
// base-2 exponential (2 ulp), with fp32 sums.  2048 x 151936 bf16: 103 us (0.89 of the
// measured copy rate; issue slots 69 % busy), with 8 alternatives 113 us (0.81), the
// gradient 202 to 206 us (0.89 to 0.91); one row with 20 alternatives 8.7 us, all
// latency.  A cluster of CTAs splits a row when there are few rows; the parts meet in distributed shared memory in rank
// order (no atomics on results: equal calls give equal bits).
//
// t is clamped to [-200, ..]: 2^t is 0 there, and 0 t stays 0 for logits of -inf
// or the type's lowest value.  NaN passes the clamp and makes S NaN.
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>
#include <set>
#include <type_traits>
#include <utility>

#include "common.cuh"
#include "internal.h"
#include "launch.h"
#include "tc_ptx.cuh"
#include "vec8.cuh"

namespace dspark {

namespace {

constexpr int GT = 256;  // threads of the gradient kernel
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kMaxTemp = 1e35f;
constexpr int kMaxSplit = 16;

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------
struct RowMeta {
  int tok;  // -1: none
  float T;
};

// what the buffers hold for row i (loads that nothing waits for yet)
struct RowRaw {
  int tok;
  float T;
  bool bad;
};
__device__ __forceinline__ RowRaw row_raw(const dspark_logit_rows& r, int i) {
  int64_t at = i;
  int ti = i;
  if (r.mark_req) {
    const int q = r.mark_req[i], pos = r.mark_pos[i];
    if (q < 0 || q >= r.n_req || pos < 0 || pos >= r.tok_cols) return RowRaw{-1, 1.f, q != -1};
    at = (int64_t)q * r.tok_cols + pos;
    ti = q;
  }
  return RowRaw{r.tokens[at], r.temp ? r.temp[ti] : 1.f, false};
}
// its token and temperature; reports what is outside its range
__device__ __forceinline__ RowMeta row_meta(const dspark_logit_rows& r, const RowRaw& raw, int i, WsHeader* hdr,
                                            bool report) {
  const bool in = raw.tok >= 0 && raw.tok < r.V;
  if ((raw.bad || (!in && raw.tok != -1)) && report && hdr) report_error(hdr, DSPARK_BAD_INPUT, i);
  return RowMeta{in ? raw.tok : -1, raw.T > 0.f && raw.T < INFINITY ? fminf(raw.T, kMaxTemp) : 1.f};
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

// The mask of U vectors, loaded ahead of its use: vector j's bits are those from
// bit `head` (below 8) of byte j on.
template <int U>
struct MaskAhead {
  uint32_t lo[U], hi[U];
  __device__ __forceinline__ void load(const uint8_t* bytes, int j, int step, int head) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      lo[u] = bytes[j + u * step];
      hi[u] = head ? bytes[j + u * step + 1] : 0;
    }
  }
  __device__ __forceinline__ uint32_t bits(int u, int head) const { return ((lo[u] | hi[u] << 8) >> head) & 255u; }
};

// A row as vectors of 8 elements from its first boundary of 16 (fp32: 32) bytes on: elements
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
  constexpr uint32_t a = Vec8<T>::kAlign;
  s.head = min(V, (int)(((a - ((uint32_t)(uintptr_t)row & (a - 1))) & (a - 1)) / sizeof(T)));
  s.nv = (V - s.head) / 8;
  return s;
}

// the largest of a warp's values (NaN is passed over)
__device__ __forceinline__ float warp_largest(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

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

// over each n lanes of a warp (the same in all of them: a + b is b + a here)
template <int n>
__device__ __forceinline__ void merge_lanes(Stat& st, int& count, float c) {
#pragma unroll
  for (int o = n / 2; o > 0; o >>= 1) {
    const Stat b{__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.S, o),
                 __shfl_xor_sync(0xffffffffu, st.A, o)};
    stat_merge(st, b, c);
    count += __shfl_xor_sync(0xffffffffu, count, o);
  }
}

// A thread's share of a row: sums of 2^t and t 2^t with t = x c - r about a
// reference r of its own, the largest element, and the count of elements above
// the token.  Sums are pairs of fp32; U vectors are summed by themselves first
// (a vector, where U is 1): added one by one to a running sum of 2^24 times their
// size, small terms would all be lost (a peaked row of 151936: S 3e-5 too small).
// The two additions a chunk cost 1 % (2048 x 151936 bf16 102.7 against 102.0 us).
//
// r is the rounded product of an element and c, so t needs one FMA and r's
// rounding cancels where the sums are moved to the largest element (stat).  r
// rises only when an element passes it by more than kLead: rising with every new
// largest element, some lane of a warp does in most steps.  A's terms of elements
// above r cancel there against t S, to 2^-24 of up to kLead S: with a lead of 32 the
// entropy of a row whose one peak comes late was off by 2e-6 (2048 x 151936 bf16 with 8
// alternatives, normal logits: 113 us with 32, 116 with 4, 118 with 2; rows that fall
// off from the front 113.5 with all).  A product above 1e7, whose rounding could move t
// by more than 1, makes the thread `wild`: its sums are void and formed again from
// (x - largest) c.
constexpr float kLead = 4.f;
struct SumsBase {
  float c, gap, r = 0.f, limit = -INFINITY, largest = -INFINITY;
  uint64_t c2, S2 = 0, A2 = 0;
  int total = 0;
  bool wild = false;
  __device__ __forceinline__ SumsBase(float c_) : c(c_), gap(kLead / c_), c2(ptx::pack2(c_, c_)) {}
  __device__ __forceinline__ void move(float d) {  // the reference by -d
    const float f = ptx::ex2(d);
    const uint64_t d2 = ptx::pack2(d, d), f2 = ptx::pack2(f, f);
    A2 = ptx::mul2(f2, ptx::fma2(d2, S2, A2));
    S2 = ptx::mul2(f2, S2);
  }
  __device__ __forceinline__ void raise(float x) {
    const float to = x * c;
    move(fminf(fmaxf(r - to, -200.f), 0.f));  // (above 0 only the first time, with nothing to move)
    r = to;
    limit = x + gap;
    wild |= fabsf(to) > 1e7f || fabsf(x) > 1e38f;
  }
  __device__ __forceinline__ void single(float x) {
    const float t = ptx::max_nan(fmaf(x, c, -r), -200.f), e = ptx::ex2(t);
    S2 = ptx::add2(S2, ptx::pack2(e, 0.f));
    A2 = ptx::add2(A2, ptx::pack2(e * t, 0.f));
    largest = fmaxf(largest, x);
  }
  // elements of a wild thread, into sums of their own
  template <int n>
  __device__ __forceinline__ void again(const float (&x)[n], float& s, float& a) const {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float t = shifted(x[i], largest, c), e = ptx::ex2(t);
      s += e;
      a = fmaf(e, t, a);
    }
  }
  __device__ __forceinline__ void join(float s, float a) {
    S2 = ptx::add2(S2, ptx::pack2(s, 0.f));
    A2 = ptx::add2(A2, ptx::pack2(a, 0.f));
  }
  // the sums about the largest element
  __device__ __forceinline__ Stat stat() {
    if (largest > -INFINITY && !wild) move(fmaf(-c, largest, r));
    const float2 s = ptx::unpack2(S2), a = ptx::unpack2(A2);
    return Stat{fmaxf(largest, kLowest), s.x + s.y, a.x + a.y};
  }
};
template <typename T>
struct Sums;
template <>
struct Sums<float> : SumsBase {
  float x_hi, x_lo, n = 0.f;
  __device__ __forceinline__ Sums(float c_, float hi, float lo) : SumsBase(c_), x_hi(hi), x_lo(lo) {}
  // U vectors; before(u): vector u lies in front of the token's.  Returns their largest element
  template <int U, typename F>
  __device__ __forceinline__ float add(const Vec8<float> (&v)[U], F before) {
    float cm = v[0].max();
#pragma unroll
    for (int u = 1; u < U; ++u) cm = fmaxf(cm, v[u].max());
    if (cm > limit) raise(cm);
    const uint64_t nr = ptx::pack2(-r, -r);
    uint64_t s2 = 0, a2 = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[8];
      v[u].get(x);
      const float xr = before(u) ? x_lo : x_hi;
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 t = ptx::unpack2(ptx::fma2(ptx::pack2(x[e], x[e + 1]), c2, nr));
        const float t0 = ptx::max_nan(t.x, -200.f), t1 = ptx::max_nan(t.y, -200.f);
        const uint64_t e2 = ptx::pack2(ptx::ex2(t0), ptx::ex2(t1));
        s2 = ptx::add2(s2, e2);
        a2 = ptx::fma2(e2, ptx::pack2(t0, t1), a2);
        n += x[e] > xr ? 1.f : 0.f;
        n += x[e + 1] > xr ? 1.f : 0.f;
      }
    }
    S2 = ptx::add2(S2, s2);
    A2 = ptx::add2(A2, a2);
    largest = fmaxf(largest, cm);
    return cm;
  }
  __device__ __forceinline__ void add_one(float x, bool before) {
    if (x > limit) raise(x);
    single(x);
    total += x > (before ? x_lo : x_hi);
  }
  __device__ __forceinline__ void flush() { total += (int)n; }  // n: below 2^24
};
template <>
struct Sums<__nv_bfloat16> : SumsBase {
  // The clamp acts on pairs before they are widened: floor is a bf16 whose t is
  // at most -200, its term 0.
  uint32_t floor2, hi2, lo2, n2 = 0;
  float x_hi, x_lo;
  // the bf16 at or below a float, in both halves
  static __device__ __forceinline__ uint32_t down2(float f) {
    const uint32_t b = __float_as_uint(f);
    return (((b & 0x80000000u) ? b + 0xFFFFu : b) >> 16) * 0x10001u;
  }
  // one below the bf16 at or below f: strictly below it whatever its size
  static __device__ __forceinline__ uint32_t under2(float f) {
    return down2(value_below<__nv_bfloat16>(__uint_as_float(down2(f) << 16)));
  }
  __device__ __forceinline__ Sums(float c_, float hi, float lo) : SumsBase(c_), x_hi(hi), x_lo(lo) {
    hi2 = down2(hi);
    lo2 = down2(lo);
    floor2 = under2(-200.f / kLead * gap);
  }
  __device__ __forceinline__ void raise(float x) {
    SumsBase::raise(x);
    floor2 = under2(x - 200.f / kLead * gap);
  }
  template <int U, typename F>
  __device__ __forceinline__ float add(const Vec8<__nv_bfloat16> (&v)[U], F before) {
    uint32_t cm2 = v[0].max2();
#pragma unroll
    for (int u = 1; u < U; ++u) cm2 = max_bf16x2(cm2, v[u].max2());
    const float cm = fmaxf(bf_lo(cm2), bf_hi(cm2));
    if (cm > limit) raise(cm);
    const uint64_t nr = ptx::pack2(-r, -r);
    uint64_t s2 = 0, a2 = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t w[4] = {v[u].a.x, v[u].a.y, v[u].a.z, v[u].a.w};
      const uint32_t xr = before(u) ? lo2 : hi2;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x = max_nan_bf16x2(w[i], floor2);
        const uint64_t t2 = ptx::fma2(ptx::pack2(bf_lo(x), bf_hi(x)), c2, nr);
        const float2 t = ptx::unpack2(t2);
        const uint64_t e2 = ptx::pack2(ptx::ex2(t.x), ptx::ex2(t.y));
        s2 = ptx::add2(s2, e2);
        a2 = ptx::fma2(e2, t2, a2);
      }
      // masks are -1 in a half; their plain sum keeps both counts (see flush)
      n2 += gt_bf16x2(w[0], xr) + gt_bf16x2(w[1], xr);
      n2 += gt_bf16x2(w[2], xr) + gt_bf16x2(w[3], xr);
    }
    S2 = ptx::add2(S2, s2);
    A2 = ptx::add2(A2, a2);
    largest = fmaxf(largest, cm);
    return cm;
  }
  __device__ __forceinline__ void add_one(float x, bool before) {
    if (x > limit) raise(x);
    single(x);
    total += x > (before ? x_lo : x_hi);
  }
  // with L masks in the low halves and H in the high ones (below 2^15 each: a
  // thread meets at most DSPARK_MAX_VOCAB / (2 LT) + 1 of either) n2 is
  // 65535 L - 65536 H = 65536 (L - H) - L
  __device__ __forceinline__ void flush() {
    const int L = (int)((0u - n2) & 0xFFFFu);
    const int diff = (int)(n2 + (uint32_t)L) >> 16;
    total += 2 * L - diff;
  }
};

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

template <int LT>
struct LpShared {
  Stat st[LT / 32];
  int cnt[LT / 32];
  // the CTA's results, read by rank 0 of the cluster
  Stat part;
  int part_cnt;
};
// The first K candidates of a CTA's part of the row, with next to no work in
// the pass over it: every thread writes down the largest element of each group
// of its vectors.  K elements reach the smallest of the w full warps' (K / w)-th
// largest threads, so only groups that reach it hold candidates; they (some 2 K of
// up to 8192) are read again.  Offering elements to a running threshold in the pass
// itself cost 49 us more than no alternatives at 2048 x 151936 bf16; this costs 11
// (with half as many groups 12: 48 MB were read again).
constexpr int kGroupBytes = 64;  // of a thread's groups: their largest elements, in the logits' type
template <int LT>
struct TopShared {
  uint64_t list[32];   // descending, 0 past the last
  uint64_t thr;        // the cluster's lower bound
  int n;               // candidates met (those past kCap were dropped)
  int picked;
  float jth[LT / 32];
  uint32_t group[kGroupBytes / 4 * LT];
};
// the place of the ring after the pass
template <int LT>
struct TopBuffer {
  static constexpr int kCap = LT * 8;  // one vector a thread always fits
  uint64_t key[kCap];           // candidates not yet in the list
  uint16_t pick[kGroupBytes / 2 * LT];  // groups to read again
};
template <int LT>
struct TopSearch {
  static constexpr int kCap = TopBuffer<LT>::kCap;
  TopShared<LT>* s;
  TopBuffer<LT>* b;
  // a key that belongs to the buffer
  __device__ __forceinline__ void offer(uint64_t key) const {
    const int at = atomicAdd(&s->n, 1);
    if (at < kCap) b->key[at] = key;
  }
  // Many keys (a short row, or a mask that leaves a few warps' threads all the
  // candidates): a bound from the keys themselves, made as the threads' was,
  // keeps some 2 K of them.  600 x 151936 with 960 candidates, 20 alternatives: 61
  // against 145 us.
  __device__ __forceinline__ int thin(int listed, int n, int K) const {
    constexpr int kMine = (kCap + LT - 1) / LT, LW = LT / 32;
    const int m = listed + n, lane = threadIdx.x & 31;
    uint64_t key[kMine], best = 0;
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      const int at = threadIdx.x + q * LT;
      key[q] = at < listed ? s->list[at] : at < m ? b->key[at - listed] : 0;
      best = key[q] > best ? key[q] : best;
    }
    float mine = best ? key_logit(best) : -INFINITY, jth = -INFINITY;
    for (int j = (K + LW - 1) / LW; j > 0; --j) {
      jth = warp_largest(mine);
      const unsigned at = __ballot_sync(0xffffffffu, mine == jth);
      if (lane == __ffs(at) - 1) mine = -INFINITY;
    }
    if (lane == 0) s->jth[threadIdx.x >> 5] = jth;
    __syncthreads();
    if (threadIdx.x == 0) s->n = 0;
    if (threadIdx.x < 32) s->list[threadIdx.x] = 0;
    float kth = s->jth[0];
#pragma unroll
    for (int w = 1; w < LW; ++w) kth = fminf(kth, s->jth[w]);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kMine; ++q)
      if (key[q] && key_logit(key[q]) >= kth) offer(key[q]);
    __syncthreads();
    return s->n;
  }
  // take with kMine keys a thread
  template <int kMine>
  __device__ __forceinline__ void place(int listed, int n) const {
    const int m = listed + n;
    uint64_t key[kMine];
    int place[kMine];
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      const int at = threadIdx.x + q * LT;
      key[q] = at < listed ? s->list[at] : at < m ? b->key[at - listed] : 0;
      place[q] = 0;
    }
#pragma unroll
    for (int q0 = 0; q0 < kMine; q0 += 2) {
      if (q0 * LT >= m) break;
#pragma unroll 4
      for (int o = 0; o < m; ++o) {
        const uint64_t other = o < listed ? s->list[o] : b->key[o - listed];
#pragma unroll
        for (int q = q0; q < min(q0 + 2, kMine); ++q) place[q] += other > key[q];
      }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kMine; ++q)
      if (key[q] && place[q] < 32) s->list[place[q]] = key[q];
  }
  // the list from `listed` keys of the list and n of the buffer, 2 LT together: a
  // key's place is the number of larger ones (keys differ).  All threads, after a barrier;
  // ends with one.
  __device__ __noinline__ void take(int listed, int n) const {
    const int m = listed + n;
    if (m <= LT) {
      // 2^sh threads count for one key
      const int sh = m <= LT / 8 ? 3 : m <= LT / 4 ? 2 : m <= LT / 2 ? 1 : 0;
      const int at = threadIdx.x >> sh, from = threadIdx.x & ((1 << sh) - 1);
      const uint64_t key = at < listed ? s->list[at] : at < m ? b->key[at - listed] : 0;
      int place = 0;
#pragma unroll 4
      for (int o = from; o < listed; o += 1 << sh) place += s->list[o] > key;
#pragma unroll 4
      for (int o = from; o < n; o += 1 << sh) place += b->key[o] > key;
      for (int d = 1; d < (1 << sh); d <<= 1) place += __shfl_xor_sync(0xffffffffu, place, d);
      __syncthreads();
      if (key && from == 0 && place < 32) s->list[place] = key;
    } else {
      place<2>(listed, n);
    }
    if (threadIdx.x == 0) s->n = 0;
    __syncthreads();
  }
  // take for any number of keys
  static __device__ __noinline__ void take_many(TopShared<LT>* s, TopBuffer<LT>* b, int listed, int n, int K) {
    const TopSearch<LT> t{s, b};
    if (listed + n <= kCap) {
      n = t.thin(listed, n, K);
      listed = 0;
    }
    if (listed + n <= 2 * LT)
      t.place<2>(listed, n);
    else
      t.place<(kCap + 32 + LT - 1) / LT>(listed, n);
    if (threadIdx.x == 0) s->n = 0;
    __syncthreads();
  }
  __device__ __forceinline__ void take_any(int listed, int n, int K) const {
    if (listed + n <= 2 * LT)
      take(listed, n);
    else
      take_many(s, b, listed, n, K);
  }
};

// A CTA's ring: chunks of U vectors of a thread (16 KB with 256 threads, 8 KB with 128)
constexpr int kMaxStages = 3, kTopStages = 2;  // 1024 threads an SM either way
template <int LT>
constexpr int kChunkBytes = 64 * LT;
constexpr long long kWaitLimit = 4000000000ll;  // cycles: about two seconds
template <typename T>
constexpr int chunk_vectors() {
  return 64 / (8 * (int)sizeof(T));
}
static_assert(sizeof(TopBuffer<128>) <= kTopStages * kChunkBytes<128> &&
                  sizeof(TopBuffer<256>) <= kTopStages * kChunkBytes<256>,
              "the buffer takes the ring's place");

template <typename T, bool kMask, bool kTop, int LT>
__global__ void __launch_bounds__(LT, 1024 / LT)
    k_logprobs(const dspark_token_logprobs_args p, WsHeader* hdr, int split) {
  constexpr int U = chunk_vectors<T>(), LW = LT / 32, CB = kChunkBytes<LT>;
  constexpr int kKeys = (kMaxSplit * 32 + LT - 1) / LT;
  constexpr int kVec = 8 * sizeof(T);
  const dspark_logit_rows& r = p.rows;
  const int i = blockIdx.x / split, rank = blockIdx.x % split;
  ptx::grid_wait();
  if (r.n_rows && i >= *r.n_rows) return;  // the whole cluster
  __shared__ LpShared<LT> sh;
  // a ring of chunks; with alternatives a TopShared after it and a TopBuffer in its place later
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages];
  __shared__ int abort_s, never_s;
  constexpr int stages = kTop ? kTopStages : kMaxStages;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* row = static_cast<const T*>(r.logits) + (int64_t)i * r.ld;
  const uint32_t* mask = kMask ? r.mask + (int64_t)i * r.mask_ld : nullptr;
  const RowShape shp = row_shape(row, r.V);
  const int v0 = (int)((int64_t)shp.nv * rank / split), v1 = (int)((int64_t)shp.nv * (rank + 1) / split);
  const T* base = row + shp.head;
  const auto load = [&](Vec8<T>& raw, int j) {
    raw.load_aligned(base + 8 * (int64_t)j);
    if (kMask) raw.mask(mask8(mask, shp.head + 8 * j));
  };
  const RowRaw given_row = row_raw(r, i);  // on its way before the ring is set up
  // one thread keeps the ring filled by bulk copies; the first chunks are under
  // way while the row's token and temperature are read
  const int chunks = (v1 - v0 + U * LT - 1) / (U * LT);
  const uint64_t policy = ptx::policy_evict_first();
  const auto fill = [&](int ch) {
    const int j0 = v0 + ch * U * LT, s = ch % stages;
    const uint32_t bytes = (uint32_t)min(U * LT, v1 - j0) * kVec;
    ptx::mbar_expect_tx(&full[s], bytes);
    ptx::bulk_load(dyn + s * CB, base + 8 * (int64_t)j0, bytes, &full[s], policy);
  };
  if (tid == 0) {
    for (int q = 0; q < stages; ++q) {
      ptx::mbar_init(&full[q], 1);
      ptx::mbar_init(&empty[q], LW);
    }
    ptx::fence_mbar_init();
    abort_s = never_s = 0;
    for (int ch = 0; ch < min(chunks, stages); ++ch) fill(ch);
  }
  __syncthreads();
  const RowMeta meta = row_meta(r, given_row, i, hdr, tid == 0 && rank == 0);
  const float c = log2_scale(meta.T);

  // rank: x > x_hi counts from the token's vector on, x > x_lo (x >= x_token) before it
  const bool given = meta.tok >= 0 && mask_bit(mask, meta.tok);
  const float xt = given ? to_f32(row[meta.tok]) : -INFINITY;
  const bool has = given && !(xt == -INFINITY);
  const int tok_vec = has ? (meta.tok < shp.head ? -1 : (meta.tok - shp.head) / 8) : -1;
  // equal elements in front of the token in its own vector
  int ties = 0;
  if (has && tok_vec >= 0 && tok_vec < shp.nv && rank == 0 && tid < 8) {
    const int v = shp.head + 8 * tok_vec + tid;
    ties = v < meta.tok && mask_bit(mask, v) && to_f32(row[v]) == xt;
  }
  Sums<T> sum(c, has ? xt : INFINITY, has ? value_below<T>(xt) : INFINITY);

  constexpr int kCap = TopBuffer<LT>::kCap, kGroups = kGroupBytes / (int)sizeof(T);
  const TopSearch<LT> top{reinterpret_cast<TopShared<LT>*>(dyn + kTopStages * CB), reinterpret_cast<TopBuffer<LT>*>(dyn)};
  // a group: 2^gshift chunks of a thread
  int gshift = 0;
  while ((chunks + (1 << gshift) - 1) >> gshift > kGroups) ++gshift;
  float gmax = -INFINITY;
  T* group = reinterpret_cast<T*>(top.s->group) + tid;
  int left = 1 << gshift;
  int stage = 0;
  uint32_t parity = 0;
  // bf16: the next whole chunk's mask is on its way while a chunk is worked on
  // (2100 x 151936, 8 alternatives: 144 against 152 us; fp32 gains nothing)
  constexpr bool kAhead = kMask && std::is_same<T, __nv_bfloat16>::value;
  const uint8_t* mask_bytes = reinterpret_cast<const uint8_t*>(mask);
  MaskAhead<U> ahead_mask;
  if (kAhead && v0 + U * LT <= v1) ahead_mask.load(mask_bytes, v0 + tid, LT, shp.head);
  for (int chunk = 0; chunk < chunks; ++chunk) {
    // refill the place of the chunk before this one
    if (tid == 0 && chunk > 0 && chunk - 1 + stages < chunks) {
      const int q = stage == 0 ? stages - 1 : stage - 1;
      if (!ptx::mbar_wait_cycles(&empty[q], stage == 0 ? parity ^ 1 : parity, &abort_s, kWaitLimit)) {
        if (hdr) report_error(hdr, DSPARK_TIMEOUT, i);
        abort_s = 1;
      }
      fill(chunk - 1 + stages);
    }
    __syncwarp();
    if (!ptx::mbar_wait_cycles(&full[stage], parity, &abort_s, kWaitLimit)) {
      if (hdr) report_error(hdr, DSPARK_TIMEOUT, i);
      abort_s = 1;
    }
    const int j = v0 + chunk * U * LT + tid;
    const uint8_t* at = dyn + stage * CB + tid * kVec;
    const int j0 = v0 + chunk * U * LT;
    float cm = -INFINITY;
    if (j0 + U * LT <= v1) {
      Vec8<T> raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        raw[u].load_shared(at + u * LT * kVec);
        if (kMask) raw[u].mask(kAhead ? ahead_mask.bits(u, shp.head) : mask8(mask, shp.head + 8 * (j + u * LT)));
      }
      if (kAhead && j0 + 2 * U * LT <= v1) ahead_mask.load(mask_bytes, j + U * LT, LT, shp.head);
      // only the token's own chunk has vectors on both sides
      if (tok_vec < j0 || tok_vec >= j0 + U * LT)
        cm = sum.add(raw, [&](int) { return tok_vec > j0; });
      else
        cm = sum.add(raw, [&](int u) { return j + u * LT < tok_vec; });
    } else {
#pragma unroll 1
      for (int u = 0; j0 + u * LT < v1; ++u) {
        Vec8<T> raw[1];
        if (j + u * LT < v1) {
          raw[0].load_shared(at + u * LT * kVec);
          if (kMask) raw[0].mask(mask8(mask, shp.head + 8 * (j + u * LT)));
        } else {
          raw[0].fill_neg_inf();
        }
        cm = fmaxf(cm, sum.add(raw, [&](int) { return j + u * LT < tok_vec; }));
      }
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&empty[stage]);
    if (++stage == stages) stage = 0, parity ^= 1;
    if (kTop) {
      gmax = fmaxf(gmax, cm);
      if (--left == 0) {
        *group = from_f32<T>(gmax);
        group += LT;
        gmax = -INFINITY;
        left = 1 << gshift;
      }
    }
  }
  // after a failure: no copy may be in flight when the CTA leaves
  if (tid == 0 && *(volatile int*)&abort_s)
    for (int ch = max(0, chunks - stages); ch < chunks; ++ch)
      ptx::mbar_wait_cycles(&full[ch % stages], (ch / stages) & 1, &never_s, kWaitLimit);
  __syncwarp();
  const int groups = (chunks + (1 << gshift) - 1) >> gshift;
  if (kTop && left < 1 << gshift) *group = from_f32<T>(gmax);
  sum.flush();
  // the elements outside the vectors, one a thread
  const bool edge = rank == 0 && tid < shp.n_edge();
  const int edge_v = edge ? shp.edge(tid) : 0;
  float edge_x = -INFINITY;
  if (edge) {
    if (mask_bit(mask, edge_v)) edge_x = to_f32(row[edge_v]);
    sum.add_one(edge_x, edge_v < meta.tok);
  }

  // warp, CTA
  if (sum.wild) {
    sum.S2 = sum.A2 = 0;
    for (int j0 = v0 + tid; j0 < v1; j0 += U * LT) {
      float s = 0.f, a = 0.f;
#pragma unroll 1
      for (int j = j0; j < min(j0 + U * LT, v1); j += LT) {
        Vec8<T> raw;
        float x[8];
        load(raw, j);
        raw.get(x);
        sum.again(x, s, a);
      }
      sum.join(s, a);
    }
    if (edge) {
      float s = 0.f, a = 0.f;
      sum.again({edge_x}, s, a);
      sum.join(s, a);
    }
  }
  Stat st = sum.stat();
  float mine = sum.largest;
  if (kTop) {
    // by the warps whose threads all have elements (a short row leaves others empty)
    const int full_warps = max(1, min(LW, (v1 - v0) / 32));
    float best = mine, jth = INFINITY;
    for (int n = warp < full_warps ? (p.top + full_warps - 1) / full_warps : 0; n > 0; --n) {
      jth = warp_largest(best);
      const unsigned at = __ballot_sync(0xffffffffu, best == jth);
      if (lane == __ffs(at) - 1) best = -INFINITY;
    }
    if (lane == 0) top.s->jth[warp] = jth;
    if (tid < 32) top.s->list[tid] = 0;
    if (tid == 0) top.s->n = top.s->picked = 0;
  }
  int ahead = sum.total + ties;
  merge_lanes<32>(st, ahead, c);
  if (lane == 0) {
    sh.st[warp] = st;
    sh.cnt[warp] = ahead;
  }
  __syncthreads();
  if (warp == 0) {
    st = sh.st[lane % LW];
    ahead = sh.cnt[lane % LW];
    merge_lanes<LW>(st, ahead, c);
  }

  if (kTop) {
    float kth = top.s->jth[0];
#pragma unroll
    for (int w = 1; w < LW; ++w) kth = fminf(kth, top.s->jth[w]);
    kth = fmaxf(kth, lowest<T>());
    if (mine >= kth) {
      for (int g = 0; g < groups; ++g)
        if (to_f32(reinterpret_cast<const T*>(top.s->group)[g * LT + tid]) >= kth) top.b->pick[atomicAdd(&top.s->picked, 1)] = (uint16_t)(g * LT + tid);
      if (edge_x >= kth) top.offer(order_key(edge_x, edge_v));
    }
    __syncthreads();
    // 2^esh vectors a group
    const int esh = (U == 4 ? 2 : 1) + gshift, items = top.s->picked << esh;
    for (int it0 = tid; it0 < items; it0 += 2 * LT) {
      Vec8<T> again[2];
      int at_j[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int it = it0 + u * LT;
        at_j[u] = v1;
        if (it < items) {
          const int g = top.b->pick[it >> esh];
          at_j[u] = v0 + (((g / LT) << esh) + (it & ((1 << esh) - 1))) * LT + g % LT;
          if (at_j[u] < v1) load(again[u], at_j[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (at_j[u] < v1)
          for (uint32_t bits = again[u].reach(kth); bits; bits &= bits - 1) {
            const int at = __ffs(bits) - 1;
            top.offer(order_key(again[u].at(at), shp.head + 8 * at_j[u] + Vec8<T>::element(at)));
          }
    }
    __syncthreads();
    const int n = top.s->n;
    if (n <= kCap) {
      top.take_any(0, n, p.top);
    } else {
      // more ties with the bound than the buffer holds: the row in steps of a
      // vector a thread, each against the list so far
      __syncthreads();
      if (tid == 0) top.s->n = 0;
      __syncthreads();
      if (edge && edge_x >= kth) top.offer(order_key(edge_x, edge_v));
      __syncthreads();
      top.take_any(0, top.s->n, p.top);
      for (int j0 = v0; j0 < v1; j0 += LT) {
        const int j = j0 + tid;
        const uint64_t last = top.s->list[p.top - 1];
        if (j < v1) {
          Vec8<T> again;
          load(again, j);
          for (uint32_t bits = again.reach(kth); bits; bits &= bits - 1) {
            const int at = __ffs(bits) - 1;
            const uint64_t key = order_key(again.at(at), shp.head + 8 * j + Vec8<T>::element(at));
            if (key > last) top.offer(key);
          }
        }
        __syncthreads();
        top.take_any(32, top.s->n, p.top);
      }
    }
  }

  if (split > 1) {
    if (tid == 0) {
      sh.part = st;
      sh.part_cnt = ahead;
      if (kTop) top.s->thr = top.s->list[p.top - 1];
    }
    __syncwarp();
    ptx::cluster_sync();
    if (rank == 0) {
      if (warp == 0) {
        // a lane each reads a CTA's part (both halves of the warp the same)
        const int q = lane % kMaxSplit;
        st = Stat{kLowest, 0.f, 0.f};
        ahead = 0;
        if (q < split) {
          st = Stat{ptx::ld_cluster_f32(ptx::map_to_rank(&sh.part.m, q)),
                    ptx::ld_cluster_f32(ptx::map_to_rank(&sh.part.S, q)),
                    ptx::ld_cluster_f32(ptx::map_to_rank(&sh.part.A, q))};
          ahead = __float_as_int(ptx::ld_cluster_f32(ptx::map_to_rank(&sh.part_cnt, q)));
        }
        __syncwarp();
        merge_lanes<kMaxSplit>(st, ahead, c);
      }
      if (kTop) {
        // the other CTAs' lists are candidates; no key below some CTA's K-th can matter
        uint64_t key[kKeys];
#pragma unroll
        for (int q = 0; q < kKeys; ++q) {
          const int o = tid + q * LT;
          key[q] = o >= 32 && o < 32 * split ? ptx::ld_cluster_u64(ptx::map_to_rank(&top.s->list[o & 31], o >> 5)) : 0;
          if ((o & 31) == p.top - 1)
            atomicMax(reinterpret_cast<unsigned long long*>(&top.s->thr), (unsigned long long)key[q]);
        }
        __syncthreads();
        const uint64_t thr = top.s->thr;
#pragma unroll
        for (int q = 0; q < kKeys; ++q)
          if (key[q] && key[q] >= thr) top.offer(key[q]);
        __syncthreads();
        top.take_any(32, top.s->n, p.top);
      }
      __syncwarp();
    }
    ptx::cluster_arrive_relaxed();  // the others' shared memory has been read
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
    if (lane < p.top) {
      const uint64_t key = top.s->list[lane];
      const bool found = key != 0 && !bad;
      p.top_id[(int64_t)i * p.top + lane] = found ? key_id(key) : -1;
      p.top_logprob[(int64_t)i * p.top + lane] =
          bad ? NAN : found ? __fdiv_rn(key_logit(key) - st.m, meta.T) - logS : -INFINITY;
    }
  }
  if (split > 1) {
    __syncwarp();
    ptx::cluster_wait();
  }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(GT, 4) k_logprobs_grad(const dspark_token_logprobs_grad_args p, WsHeader* hdr,
                                                         int split) {
  constexpr int U = std::is_same<T, float>::value ? 2 : 4;
  const dspark_logit_rows& r = p.rows;
  const int i = blockIdx.x / split, rank = blockIdx.x % split;
  ptx::grid_wait();
  if (r.n_rows && i >= *r.n_rows) return;  // the whole cluster
  __shared__ int pid[DSPARK_MAX_TOP + 1];
  __shared__ float pg[DSPARK_MAX_TOP + 1], px[DSPARK_MAX_TOP + 1];
  const int tid = threadIdx.x;
  const RowMeta meta = row_meta(r, row_raw(r, i), i, hdr, tid == 0 && rank == 0);
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
  const bool vec = ((uintptr_t)obase & (Vec8<T>::kAlign - 1)) == 0;
  for (int j0 = v0; j0 < v1; j0 += U * GT) {
    Vec8<T> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * GT + tid;
      if (j < v1) raw[u].load_aligned(base + 8 * (int64_t)j);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * GT + tid;
      if (j >= v1) continue;
      float x[8];
      if (mask) raw[u].mask(mask8(mask, shp.head + 8 * j));
      raw[u].get(x);
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

// CTAs a row is split over: about as many as have a place at once, each with
// `least` elements or more (8192, but 4096 where rows are very few: 1 x 100003 fp32 with
// a mask 9.2 us, with 8192 10.2; 32 x 4264 with 20 alternatives 7.5 us, with 2048
// 10.1).  V = 151936 bf16, without alternatives: 16 rows 6.0 us with 16 CTAs a row (8:
// 6.2), 32 rows 6.7 with 8 (16: 7.6), 64 rows 9.4 with 4 (8: 10.8), 150 rows 14.4 with 2 (4: 17.9), 300 rows 21.9 with 1 (2: 22.9); 300 x 32000 with 8
// alternatives 11.3 with 1 (2: 15.3).  The gradient keeps fewer bytes on their way
// to a CTA and wants more of them: 64 rows 10.2 with 8 (4: 10.7), 300 rows 34.0 with 2 (1: 38.9).
int row_split(int64_t N, int64_t V, int64_t most, int64_t least) {
  int split = 1;
  while (split < kMaxSplit && N * split * 2 <= (split == 8 ? 256 : most) && V >= least * split * 2) split *= 2;
  return split;
}
constexpr int kMostLp = 400, kMostGrad = 608, kLeast = 2048;

// Clusters of 16 CTAs: the attribute belongs to the kernel in a device's
// context, so it is set once per (device, kernel).
cudaError_t allow_large_cluster(const void* kernel) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::mutex mu;
  static std::set<std::pair<int, const void*>> done;
  std::lock_guard<std::mutex> lock(mu);
  if (done.count({dev, kernel})) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done.insert({dev, kernel});
  return e;
}

template <typename K, typename A>
cudaError_t launch_rows(K kernel, const A& a, WsHeader* hdr, int N, int split, int threads, unsigned smem,
                        cudaStream_t s) {
  if (smem > 0)
    if (const cudaError_t e = ensure_smem_limit((const void*)kernel, (int)smem); e != cudaSuccess) return e;
  if (split > 8)
    if (const cudaError_t e = allow_large_cluster((const void*)kernel); e != cudaSuccess) return e;
  const cudaError_t e = launch_overlapped(kernel, (unsigned)N * (unsigned)split, (unsigned)threads, smem,
                                          (unsigned)split, s, a, hdr, split);
  if (e != cudaSuccess) return e;
  count_launches(1);
  return cudaGetLastError();
}

template <typename T, int LT>
cudaError_t launch_logprobs(const dspark_token_logprobs_args& a, WsHeader* hdr, int split, cudaStream_t s) {
  const auto go = [&](auto kernel, unsigned smem) { return launch_rows(kernel, a, hdr, a.rows.N, split, LT, smem, s); };
  const bool mask = a.rows.mask != nullptr;
  // the ring's depth is a constant of the kernel (a run-time one: 2048 x 151936 bf16 106 against 101 us)
  if (a.top > 0) {
    const unsigned smem = kTopStages * kChunkBytes<LT> + sizeof(TopShared<LT>);
    return mask ? go(k_logprobs<T, true, true, LT>, smem) : go(k_logprobs<T, false, true, LT>, smem);
  }
  const unsigned smem = kMaxStages * kChunkBytes<LT>;
  return mask ? go(k_logprobs<T, true, false, LT>, smem) : go(k_logprobs<T, false, false, LT>, smem);
}

}  // namespace

size_t token_logprobs_ws(int, int, int) { return sizeof(WsHeader); }

cudaError_t launch_token_logprobs(const dspark_token_logprobs_args& a, uint8_t* ws, cudaStream_t s) {
  WsHeader* hdr = reinterpret_cast<WsHeader*>(ws);
  const int N = a.rows.N, split = row_split(N, a.rows.V, kMostLp, N <= 32 ? 2 * kLeast : 4 * kLeast);
  const bool bf16 = a.rows.dtype == DSPARK_BF16;
  // Many rows for their length: CTAs of 128 threads, eight an SM, so that more rows
  // cover a row's start and end.  bf16, 128 against 256 threads: 500 x 14088 with 20
  // alternatives 11.8 and 13.8 us, 2932 x 14088 35.8 and 52.2, 2047 x 64367 with 5 59.1 and
  // 64.9, 2048 x 151936 with 8 114 and 118; but 1352 x 151936 75.9 and 70.2, 100 x 1280 with 20 8.6 and 6.9
  const int64_t bytes = (int64_t)a.rows.V * (bf16 ? 2 : 4);
  if (N >= 200 && N * (int64_t)200 >= bytes)
    return bf16 ? launch_logprobs<__nv_bfloat16, 128>(a, hdr, 1, s) : launch_logprobs<float, 128>(a, hdr, 1, s);
  return bf16 ? launch_logprobs<__nv_bfloat16, 256>(a, hdr, split, s) : launch_logprobs<float, 256>(a, hdr, split, s);
}

cudaError_t launch_token_logprobs_grad(const dspark_token_logprobs_grad_args& a, uint8_t* ws, cudaStream_t s) {
  WsHeader* hdr = reinterpret_cast<WsHeader*>(ws);
  const int N = a.rows.N, split = row_split(N, a.rows.V, kMostGrad, kLeast);
  return a.rows.dtype == DSPARK_BF16 ? launch_rows(k_logprobs_grad<__nv_bfloat16>, a, hdr, N, split, GT, 0, s)
                                     : launch_rows(k_logprobs_grad<float>, a, hdr, N, split, GT, 0, s);
}

}  // namespace dspark
