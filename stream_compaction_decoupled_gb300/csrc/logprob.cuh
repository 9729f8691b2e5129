// logprob.cuh -- log probabilities of given tokens from rows of logits, with the entropy
// of each row and its most likely alternatives, and the gradient.
//
//   lse = log sum exp(x_j),  logprob = x_target - lse,  p_j = exp(x_j - lse),
//   entropy = -sum p_j log p_j,  top: the K largest x_j in falling order, ties to the
//   lower index, with their log probabilities;
//   gradient:  dx_j = dlogprob ([j = target] - p_j) - dentropy p_j (log p_j + entropy).
//
// Each row is read once.  A thread keeps the largest value so far, M, and relative to it
// s = sum e^z and t = sum e^z z with z = x - M; when M grows, s and t are moved to the new
// one.  At the end
//   lse = M + log s,   entropy = log s - t / s,   logprob = (x_target - M) - log s.
// M is the true maximum: below it, a confident row's log s and t / s would both be large and
// cancel, and lse would not be the least number that it can be, M, so that e^(x - lse) could
// pass 1.  In 16-bit types the sums are kept in base 2 (LpAcc), one fused multiply-add to an
// exponent in place of a difference and a product.
// Values are held at a floor (-2^126; bf16 -2^20, fp16 its lowest), so that a masked logit
// (-inf, or a number far below) gives e^z = 0 and a product of 0, not a NaN.  Rows for which
// this does not do (nothing above the floor, values far from 0, a NaN) are read again by the
// careful form in lp_careful.
//
// The alternatives are found in the same pass, as a compaction.  A value's key (the value
// in the high half, the index reversed in the low half: unique, so ties are settled) is
// compared with a threshold that K values are known to reach: at first the K-th largest
// of 64 group maxima of the first tile.  The test is one comparison a pack of 16 bytes;
// packs that pass, a few of a tile, go to a list in shared memory, with no barrier.  The
// list is expanded into keys after tiles 2, 6, 18, ... and at the end: the K largest are
// kept, in order, and the threshold rises past the K-th, so that about K packs pass
// between one time and the next.  Where the list overflows (values that rise along the
// row), the tiles from there on are gone through again, 256 packs at a time.
//
// With few rows a cluster of CTAs shares each row, slice by slice; CTA 0 of the cluster
// reads the others' sums and lists through distributed shared memory.
//
// Rows start anywhere: packs of 16 bytes are laid over the row from the boundary below its
// first value, and values outside the row or the slice count as masked.
//
// Measured (GB300, copy rate 6.8 TB/s): 4096 x 128000 bf16 158.5 us without alternatives (6.6
// TB/s, HBM), 205 with 8 and 253 with 32 (5.1 and 4.1 TB/s, issue); 7 x 50021 fp32 with 20
// alternatives 12.6 us, the latency of threshold, selection and merge; the gradient of 4096
// x 32000 bf16 97.8 us (5.4 TB/s, half of it writes).  Rows that rise along the vocabulary, whose
// list overflows in every tile: 4096 x 32000 bf16 with 8 alternatives 911 us, where rows in no
// order take 85.
#pragma once

#include <cfloat>
#include <climits>

#include "lm.cuh"
#include "lm.h"

namespace gbs {

template <class T> struct LogprobArgs {
  const T* logits;
  long long stride;
  const void* targets;
  int targets64;
  float *logprob, *entropy, *lse, *top_values;
  int32_t* top_ids;
  int V, K;
  ErrSink err;
};

constexpr int kLpThreads = 256;
constexpr int kLpPacks = 4;        // packs of a thread in a tile
constexpr int kLpGradPacks = 4;    // and in a block of the gradient
constexpr int kLpGroups = 64;      // groups of threads whose maxima give the first threshold
constexpr int kLpStages = 2;       // tiles in shared memory
constexpr int kLpList = 256;       // packs
constexpr int kLpKeys = 1024;      // keys
constexpr int kLpMaxCluster = 8;
// Natural-log differences from a maximum stop here: e^d has long been 0 in fp32, and
// products with d stay finite, so that 0 times them is 0.
constexpr float kLpFloor = -1000.f;

__device__ __forceinline__ long long lp_target(const void* targets, int is64, long long row) {
  return is64 ? ((const long long*)targets)[row] : (long long)((const int*)targets)[row];
}

// Keys: larger value first, then lower index; 0 is below every key.  NaN counts as the
// largest value, -0 as +0.
__device__ __forceinline__ unsigned lp_order(float x) {
  unsigned u = __float_as_uint(x + 0.f);
  if (x != x) u = 0x7fc00000u;
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float lp_unorder(unsigned u) {
  return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ unsigned long long lp_key(float x, int index) {
  return (unsigned long long)lp_order(x) << 32 | (0x7fffffffu - (unsigned)index);
}

// The floor under the values of a type, and a pack held at it.
template <class T> struct LpType;
template <> struct LpType<float> {
  static constexpr float kFloor = -8.507059173023462e37f;  // -2^126
  static __device__ __forceinline__ float hold(Pack<float, 4>& p) {
#pragma unroll
    for (int c = 0; c < 4; ++c) p.v[c] = max_nan(p.v[c], kFloor);
    return max_nan(max_nan(p.v[0], p.v[1]), max_nan(p.v[2], p.v[3]));
  }
};
template <> struct LpType<__nv_bfloat16> {
  static constexpr float kFloor = -1048576.f;  // -2^20
  static __device__ __forceinline__ unsigned max2(unsigned a, unsigned b) {
    unsigned d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ float hold(Pack<__nv_bfloat16, 8>& p) {
    uint4 u;
    memcpy(&u, &p, 16);
    constexpr unsigned f = 0xc980c980u;
    u = make_uint4(max2(u.x, f), max2(u.y, f), max2(u.z, f), max2(u.w, f));
    memcpy(&p, &u, 16);
    const unsigned m = max2(max2(u.x, u.y), max2(u.z, u.w));
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
};
template <> struct LpType<__half> {
  static constexpr float kFloor = -65504.f;
  static __device__ __forceinline__ unsigned max2(unsigned a, unsigned b) {
    unsigned d;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ float hold(Pack<__half, 8>& p) {
    uint4 u;
    memcpy(&u, &p, 16);
    constexpr unsigned f = 0xfbfffbffu;
    u = make_uint4(max2(u.x, f), max2(u.y, f), max2(u.z, f), max2(u.w, f));
    memcpy(&p, &u, 16);
    const unsigned m = max2(max2(u.x, u.y), max2(u.z, u.w));
    __half2 h;
    memcpy(&h, &m, 4);
    const float2 q = __half22float2(h);
    return max_nan(q.x, q.y);
  }
};

// The largest value m, and relative to it r = sum e^z - 1 (of all values but one largest) and
// t = sum e^z z: what other threads' many small terms add to in a confident row is not lost
// beside the 1.  r = -1: no values.
struct LpSums {
  float m, r, t;
};
__device__ __forceinline__ LpSums lp_join(LpSums a, LpSums b) {
  const LpSums hi = a.m < b.m ? b : a, lo = a.m < b.m ? a : b;
  const float d = max_nan(lo.m - hi.m, kLpFloor), k = ex2(d * kLog2e), s = 1.f + lo.r;
  return {hi.m, fmaf(k, s, hi.r), fmaf(k, fmaf(s, d, lo.t), hi.t)};
}

// A thread's sums while it goes along its values, in pairs, s the whole sum.  fp32: as above.
template <class T> struct LpAcc {
  static constexpr float kFar = 1e38f;  // differences of values up to here stay finite
  float m = LpType<T>::kFloor;
  float2 s = make_float2(0.f, 0.f), t = make_float2(0.f, 0.f);
  __device__ __forceinline__ void rise(float best) {  // best > m
    const float d = max_nan(m - best, kLpFloor), k = ex2(d * kLog2e);
    move(d, k);
    m = best;
  }
  __device__ __forceinline__ void move(float d, float k) {
    const float2 k2 = make_float2(k, k);
    t = mul2(k2, fma2(s, make_float2(d, d), t));
    s = mul2(s, k2);
  }
  __device__ __forceinline__ void add(float2 v) {
    const float2 z = add2(v, make_float2(-m, -m)), y = mul2(z, make_float2(kLog2e, kLog2e));
    // Off by (2 + 1.2 |z|) units of 2^-24: |z| e^-|z| of that, 0.5 units at most, is the sum's
    // share, less than its own roundings.  (With expf: 4096 x 32000 94 us, with this 80.)
    const float2 e = make_float2(ex2(y.x), ex2(y.y));
    s = add2(s, e);
    t = fma2(e, z, t);
  }
  __device__ __forceinline__ LpSums sums() const { return {m, s.x + s.y - 1.f, t.x + t.y}; }
};
// 16 bits: relative to r = m log2(e) as rounded, in base 2, s = sum 2^d and t = sum 2^d d with
// d = x log2(e) - r exact but for one rounding (half an instruction a value less: 4096 x 128000
// bf16 with 8 alternatives 204.6 us, with differences first 213.6).  d is z log2(e) + f, f = m
// log2(e) - r: known exactly and taken out at the end.  (Further than kFar from 0 it is no small fraction any
// more; the floor, and so every thread's m, is little below that.)
template <class T> struct LpAcc16 : LpAcc<float> {
  static constexpr float kFar = 1e6f;
  float r;
  __device__ __forceinline__ LpAcc16() {
    m = LpType<T>::kFloor;
    r = m * kLog2e;
  }
  __device__ __forceinline__ void rise(float best) {
    const float to = best * kLog2e, d = max_nan(r - to, kLpFloor);
    move(d, ex2(d));
    m = best;
    r = to;
  }
  __device__ __forceinline__ void add(float2 v) {
    const float2 d = fma2(v, make_float2(kLog2e, kLog2e), make_float2(-r, -r));
    const float2 e = make_float2(ex2(d.x), ex2(d.y));
    s = add2(s, e);
    t = fma2(e, d, t);
  }
  __device__ __forceinline__ LpSums sums() const {
    // 2^-f - 1 by its series: |f| is 2^-4 at most, and the next term under 2^-22.
    const float f = fmaf(m, kLog2e, -r), x = kLn2 * f, k = -x * (1.f - x * (0.5f - x * (1.f / 6.f)));
    const float s1 = s.x + s.y, t1 = fmaf(-f, s1, t.x + t.y);
    return {m, fmaf(s1, k, s1 - 1.f), kLn2 * fmaf(t1, k, t1)};
  }
};
template <> struct LpAcc<__nv_bfloat16> : LpAcc16<__nv_bfloat16> {};
template <> struct LpAcc<__half> : LpAcc16<__half> {};

struct LpShared {
  unsigned long long keys[kLpKeys];
  uint4 list[kLpList];
  int list_at[kLpList];          // the index of each pack's first value
  uint4 again[kLpThreads];       // packs read again
  unsigned long long group[kLpGroups];
  LpSums warp[kLpThreads / 32];
  LpSums sums;                   // the CTA's
  unsigned long long tau, pivot;
  int listed, count, left;
  int missed;                    // the first tile (its first pack) that the list had no room for
};

// The CTA's sums from its threads', in a fixed order; ends with a barrier.
__device__ __forceinline__ void lp_reduce(LpSums v, LpShared& sh) {
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    LpSums o;
    o.m = __shfl_xor_sync(0xffffffffu, v.m, d);
    o.r = __shfl_xor_sync(0xffffffffu, v.r, d);
    o.t = __shfl_xor_sync(0xffffffffu, v.t, d);
    v = lp_join(v, o);
  }
  if (threadIdx.x % 32 == 0) sh.warp[threadIdx.x / 32] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    LpSums r = sh.warp[0];
    for (int w = 1; w < kLpThreads / 32; ++w) r = lp_join(r, sh.warp[w]);
    sh.sums = r;
  }
  __syncthreads();
}

// The sums of a whole row value by value: for values near the ends of the range.  A row with
// nothing left ends with r = -1.
template <class T> __device__ void lp_careful(const T* x, int V, LpShared& sh) {
  LpSums v = {-FLT_MAX, -1.f, 0.f};
  for (int j = threadIdx.x; j < V; j += kLpThreads) {
    const float q = widen(x[j]);
    v = lp_join(v, {q, q == -INFINITY ? -1.f : q - q, 0.f});  // q - q: 0, or a NaN
  }
  lp_reduce(v, sh);
}

// Of 64 groups of threads (a fixed number of neighbours each) the K-th largest of the
// groups' largest keys, or 0 where fewer than K groups have one.  All threads of the CTA
// call it; it begins with a write to shared memory and ends with a barrier.
__device__ __forceinline__ unsigned long long lp_kth_group(unsigned long long k, int K, LpShared& sh) {
  constexpr int per = kLpThreads / kLpGroups;
  const int tid = threadIdx.x;
#pragma unroll
  for (int d = 1; d < per; d *= 2) {
    const unsigned long long o = __shfl_xor_sync(0xffffffffu, k, d);
    k = o > k ? o : k;
  }
  if (tid % per == 0) sh.group[tid / per] = k;
  if (tid == 0) sh.pivot = 0;
  __syncthreads();
  int above = 0;
#pragma unroll
  for (int g = 0; g < kLpGroups; g += per) above += sh.group[g + tid % per] > k;
#pragma unroll
  for (int d = 1; d < per; d *= 2) above += __shfl_xor_sync(0xffffffffu, above, d);
  if (tid % per == 0 && above == K - 1 && k) sh.pivot = k;
  __syncthreads();
  return sh.pivot;
}

// Leaves the K largest of keys[0 .. n) first, in falling order, zeros where there are fewer.
// Many keys are first thinned: those below the K-th largest of 64 groups' largest go, which
// leaves at most K n / 64 or so.  The rest are placed by counting the larger ones.  All
// threads of the CTA call it after a barrier; ends with a barrier.
__device__ __forceinline__ void lp_select(int n, int K, LpShared& sh) {
  const int tid = threadIdx.x;
  constexpr int kMany = 128;
  while (n > kMany) {
    constexpr int M = kLpKeys / kLpThreads;
    unsigned long long mine[M], most = 0;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int at = tid + m * kLpThreads;
      mine[m] = at < n ? sh.keys[at] : 0;
      most = mine[m] > most ? mine[m] : most;
    }
    const unsigned long long pivot = lp_kth_group(most, K, sh);
    if (tid == 0) sh.left = 0;
    __syncthreads();
#pragma unroll
    for (int m = 0; m < M; ++m)
      if (mine[m] && mine[m] >= pivot) sh.keys[atomicAdd(&sh.left, 1)] = mine[m];
    __syncthreads();
    n = sh.left;
  }
  const int per = n <= 32 ? 8 : n <= 64 ? 4 : 2, at = tid / per;
  const unsigned long long mine = at < n ? sh.keys[at] : 0;
  int above = 0;
  if (at < n) {
#pragma unroll 4
    for (int j = tid % per; j < n; j += per) above += sh.keys[j] > mine;
  }
  for (int d = 1; d < per; d *= 2) above += __shfl_xor_sync(0xffffffffu, above, d);
  __syncthreads();
  if (tid >= n && tid < K) sh.keys[tid] = 0;
  if (at < n && tid % per == 0 && above < K) sh.keys[above] = mine;
  __syncthreads();
}

template <class T, bool TOP>
__global__ void __launch_bounds__(kLpThreads, 4) logprob_kernel(const __grid_constant__ LogprobArgs<T> a, unsigned C) {
  constexpr int V = 16 / sizeof(T), U = kLpPacks, NT = kLpThreads;
  constexpr float kFloor = LpType<T>::kFloor;
  static_assert(kLpStages == 2, "two tiles in turn");
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ LpShared sh;
  pdl_entry();
  const int tid = threadIdx.x;
  const unsigned rank = C > 1 ? cluster_rank() : 0;
  const long long row = blockIdx.x / C;
  const T* x = a.logits + row * a.stride;
  const int off = (int)((uintptr_t)x % 16 / sizeof(T));
  const int packs = (int)(((long long)off + a.V + V - 1) / V);
  const int per = (packs + (int)C - 1) / (int)C;
  const int p0 = (int)rank * per < packs ? (int)rank * per : packs;
  const int p1 = p0 + per < packs ? p0 + per : packs;
  const long long end_ = (long long)p1 * V - off;
  const int end = end_ < a.V ? (int)end_ : a.V;  // values of the slice end here

  if (TOP && tid == 0) {
    sh.listed = 0;
    sh.count = 0;
    sh.tau = 0;
    sh.missed = INT_MAX;
  }

  // A thread's packs of a tile, copied one tile ahead into shared memory of its own.
  auto slot = [&](int stage, int u) { return ring + ((stage * U + u) * NT + tid) * 16; };
  auto fetch = [&](int p, int stage) {
    if (p > 0 && p + U * NT < p1) {  // whole packs of the row
      const T* q = x + ((p + tid) * V - off);
#pragma unroll
      for (int u = 0; u < U; ++u) cp_async16(slot(stage, u), q + u * NT * V);
      cp_async_commit();
      return;
    }
#pragma unroll 1
    for (int u = 0; u < U; ++u) {
      const int j = p + u * NT + tid, e0 = j * V - off;
      if (j < p1 && e0 >= 0 && e0 + V <= a.V) {
        cp_async16(slot(stage, u), x + e0);
      } else if (p < p1) {  // the row's ends, and what lies past the slice
        T* dst = (T*)slot(stage, u);
#pragma unroll 1
        for (int c = 0; c < V; ++c)
          dst[c] = j < p1 && (unsigned)(e0 + c) < (unsigned)a.V ? x[e0 + c] : narrow<T>(-INFINITY);
      }
    }
    cp_async_commit();
  };
  // Expands the listed packs before index `before` into keys and empties the list; the K
  // largest are left among the keys, in order, and the threshold is past the K-th.  Called
  // after a barrier, ends with one.
  auto flush = [&](int before) {
    const int listed = sh.listed < kLpList ? sh.listed : kLpList;
    for (int q0 = 0; q0 < listed * V; q0 += kLpKeys / 2) {
      const unsigned long long tau = sh.tau;
      // A pass adds up to kLpKeys / 2 keys.  The first finds at most K; before a later one the
      // keys are thinned where there may not be room.  All threads read the count before any
      // adds to it, so that they take the same way.
      if (q0 > 0) {
        const int have = sh.count;
        __syncthreads();
        if (have > kLpKeys / 2) {
          lp_select(have, a.K, sh);
          if (tid == 0) sh.count = a.K;
          __syncthreads();
        }
      }
      for (int q = q0 + tid; q < listed * V && q < q0 + kLpKeys / 2; q += NT) {
        const int e0 = sh.list_at[q / V], i = e0 + q % V;
        const unsigned long long k = lp_key(widen(((const T*)sh.list)[q]), i);
        if (e0 < before && (unsigned)i < (unsigned)end && k >= tau) sh.keys[atomicAdd(&sh.count, 1)] = k;
      }
      __syncthreads();
    }
    const int n = sh.count;
    lp_select(n, a.K, sh);
    if (tid == 0) {
      sh.listed = 0;
      if (n >= a.K) {
        sh.count = a.K;
        sh.tau = sh.keys[a.K - 1] + 1;
      }
    }
    __syncthreads();
  };
  // Puts a pack of this thread's into the list, at q in shared memory; false: no room.
  auto put = [&](const unsigned char* q, int e0) {
    const int at = atomicAdd(&sh.listed, 1);
    if (at >= kLpList) return false;
    sh.list[at] = *(const uint4*)q;
    sh.list_at[at] = e0;
    return true;
  };
  // Whether a pack's largest key reaches the threshold.
  auto reaches = [&](const T* q, int e0) {
    float m = widen(q[0]);
#pragma unroll 1
    for (int c = 1; c < V; ++c) m = max_nan(m, widen(q[c]));
    return lp_key(m, e0 > 0 ? e0 : 0) >= sh.tau;
  };
  // Brings the keys up to date with all packs before `p`.  Called after a barrier, by all.
  auto settle = [&](int p) {
    const int from = sh.missed;
    flush(from == INT_MAX ? INT_MAX : from * V - off);
    if (from == INT_MAX) return;
    unsigned char* mine = (unsigned char*)&sh.again[tid];
    for (int j0 = from; j0 < p && j0 < p1; j0 += NT) {
      const int j = j0 + tid, e0 = j * V - off;
      if (j < p && j < p1) {
#pragma unroll 1
        for (int c = 0; c < V; ++c)
          ((T*)mine)[c] = (unsigned)(e0 + c) < (unsigned)a.V ? x[e0 + c] : narrow<T>(-INFINITY);
        if (reaches((const T*)mine, e0)) put(mine, e0);  // the list is empty: there is room
      }
      __syncthreads();
      flush(INT_MAX);
    }
    if (tid == 0) sh.missed = INT_MAX;
    __syncthreads();
  };
  LpAcc<T> acc;
  float bar = -INFINITY;  // the threshold's value
  int stage = 0, tile = 1, next = 2;
  fetch(p0, 0);
  long long target = -1;
  float xt = 0.f;
  if (rank == 0 && tid == 0) {
    target = lp_target(a.targets, a.targets64, row);
    if (target >= a.V) {  // no such token: reported, and treated as ignored
      raise_err(a.err, ERRBIT_RANGE);
      target = -1;
    }
    if (target >= 0) xt = widen(x[target]);
  }
  for (int p = p0; p < p1; p += U * NT, ++tile) {
    fetch(p + U * NT, stage ^ 1);
    cp_async_wait<1>();
    float bests[U];                   // the largest value of each pack, or the floor
    unsigned long long most = 0;      // first tile: a key that some value here reaches
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Pack<T, V> held = ld_pack<T, V>((const T*)slot(stage, u));
      const float best = bests[u] = LpType<T>::hold(held);
      if (TOP && p == p0) {
        // A pack is known to hold a value of at least its largest (the floor may stand for
        // -inf) at an index no later than its last.
        const int j = p + u * NT + tid;
        int i = j * V - off + V - 1;
        if (i >= end) i = end - 1;
        const unsigned long long q = j < p1 ? lp_key(best <= kFloor ? -INFINITY : best, i) : 0;
        most = q > most ? q : most;
      }
      if (best > acc.m) acc.rise(best);
      float v[V];
      widen_pack(held, v);
#pragma unroll
      for (int c = 0; c < V; c += 2) acc.add(make_float2(v[c], v[c + 1]));
    }
    if constexpr (TOP) {
      if (p == p0) {
        const unsigned long long kth = lp_kth_group(most, a.K, sh);
        if (tid == 0) sh.tau = kth;
        __syncthreads();
        bar = sh.tau ? lp_unorder((unsigned)(sh.tau >> 32)) : -INFINITY;
      }
      float tallest = bests[0];
#pragma unroll
      for (int u = 1; u < U; ++u) tallest = max_nan(tallest, bests[u]);
      if (!(tallest < bar)) {
        // Packs past the threshold's value, and those perhaps level with it.
        unsigned over = 0, even = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (bests[u] > bar && bests[u] > kFloor) over |= 1u << u;
          else if (!(bests[u] < bar)) even |= 1u << u;  // the floor may stand for -inf
        }
#pragma unroll 1
        for (unsigned left = over | even; left; left &= left - 1) {
          const int u = __ffs(left) - 1, j = p + u * NT + tid, e0 = j * V - off;
          const unsigned char* q = slot(stage, u);
          if (j >= p1 || (even >> u & 1 && !reaches((const T*)q, e0))) continue;
          if (!put(q, e0)) atomicMin(&sh.missed, p);
        }
      }
      if (tile == next && p + U * NT < p1) {
        next *= 3;
        __syncthreads();
        settle(p + U * NT);
        bar = sh.tau ? lp_unorder((unsigned)(sh.tau >> 32)) : -INFINITY;
      }
    }
    stage ^= 1;
  }
  lp_reduce(acc.sums(), sh);
  if constexpr (TOP) settle(INT_MAX);
  if (C > 1) {
    cluster_sync();
    if (rank == 0) {
      if (tid == 0) {
        LpSums r = sh.sums;
        for (unsigned q = 1; q < C; ++q) {
          const unsigned at = cluster_addr(&sh.sums, q);
          r = lp_join(r, {ld_cluster_f32(at), ld_cluster_f32(at + 4), ld_cluster_f32(at + 8)});
        }
        sh.sums = r;
      }
      if constexpr (TOP) {
        for (int i = a.K + tid; i < (int)C * a.K; i += NT)
          sh.keys[i] = ld_cluster_u64(cluster_addr(&sh.keys[i % a.K], (unsigned)(i / a.K)));
        __syncthreads();
        lp_select((int)C * a.K, a.K, sh);
      }
      __syncthreads();
    }
    cluster_sync();  // the others' shared memory has been read
    if (rank != 0) return;
  }
  LpSums r = sh.sums;
  // Nothing above the floor, a maximum far from 0, or a NaN: read the row again with care.
  // (The same for all threads.)
  if (!(r.m > kFloor) || !(fabsf(r.m) < LpAcc<T>::kFar) || !(r.r < INFINITY)) {
    __syncthreads();
    lp_careful(x, a.V, sh);
    r = sh.sums;
  }
  const float log_s = log1pf(r.r);
  auto logprob = [&](float v) { return (v - r.m) - log_s; };
  const bool none = r.r == -1.f;  // all -inf
  if (tid == 0) {
    a.lse[row] = none ? -INFINITY : r.m + log_s;
    a.entropy[row] = none ? 0.f : log_s - r.t / (1.f + r.r);
    a.logprob[row] = target < 0 ? 0.f : none ? -INFINITY : logprob(xt);
  }
  if constexpr (TOP) {
    if (tid < a.K) {
      const unsigned long long k = sh.keys[tid];
      a.top_ids[row * a.K + tid] = (int32_t)(0x7fffffffu - (unsigned)k);
      a.top_values[row * a.K + tid] = none ? -INFINITY : logprob(lp_unorder((unsigned)(k >> 32)));
    }
  }
}

// The gradient: one read and one write of each logit, U packs a thread,
//   dx = -p (w + h (log p + entropy)),   p = exp(x - lse),   and w more at the target
// (w = dlogprob, h = dentropy).  Values are held at a floor far below any lse but small
// enough that its products stay finite, so that a masked logit gets 0; rows whose lse is
// itself near the floor (or -inf, or NaN), or as far above 0, or whose h is that large, take
// each difference with care instead.  Where
// the rows of the two arrays start at different offsets from a 16-byte boundary V is 1.
template <class T> struct LogprobGradArgs {
  const T* logits;
  T* dlogits;
  long long stride, dstride;
  const void* targets;
  int targets64;
  const float *lse, *entropy, *dlogprob, *dentropy;
  int V, blocks;  // blocks of a row
};

// A pack held at the gradient's floor: -2^66 (fp16: its lowest).
template <class T, int V> __device__ __forceinline__ void lp_grad_hold(Pack<T, V>& p) {
  if constexpr (V == 8) {
    uint4 u;
    memcpy(&u, &p, 16);
    constexpr unsigned f = std::is_same<T, __half>::value ? 0xfbfffbffu : 0xe080e080u;
    u = make_uint4(LpType<T>::max2(u.x, f), LpType<T>::max2(u.y, f), LpType<T>::max2(u.z, f), LpType<T>::max2(u.w, f));
    memcpy(&p, &u, 16);
  } else {
    const float f = std::is_same<T, __half>::value ? -65504.f : -7.378697629483821e19f;
#pragma unroll
    for (int c = 0; c < V; ++c) p.v[c] = narrow<T>(max_nan(widen(p.v[c]), f));
  }
}

// e^d.  2^(d log2 e) with the product rounded once is off by up to 8, 15 and 31 units of 2^-24 at
// d = -10, -20 and -40: a 16-bit output's own rounding (2^-9 or 2^-12) hides that, fp32's not.
template <class T> __device__ __forceinline__ float2 lp_exp(float2 d) {
  if constexpr (sizeof(T) == 4) return exp_full(d);
  const float2 y = mul2(d, make_float2(kLog2e, kLog2e));
  return make_float2(ex2(y.x), ex2(y.y));
}

// fp32: six CTAs an SM, 40 registers (4096 x 32000, 16384 x 4096, 8192 x 1000: 148, 97 and 24.7
// us; five 154, 105, 24.8; eight 150, 94, 25.9).  16 bits: as the compiler has it, 44.
template <class T, int V>
__global__ void __launch_bounds__(kLpThreads, sizeof(T) == 4 ? 6 : 0) logprob_backward_kernel(const __grid_constant__ LogprobGradArgs<T> a) {
  constexpr int U = kLpGradPacks, NT = kLpThreads;
  pdl_entry();
  const long long row = blockIdx.x / a.blocks;
  const T* x = a.logits + row * a.stride;
  T* dx = a.dlogits + row * a.dstride;
  const int off = V == 1 ? 0 : (int)((uintptr_t)x % 16 / sizeof(T));
  const int first = ((int)(blockIdx.x % a.blocks) * U * NT + threadIdx.x) * V - off;
  // All of the row's numbers at once: none waits for another.
  const long long target = lp_target(a.targets, a.targets64, row);
  const float lse = a.lse[row], dl = a.dlogprob ? a.dlogprob[row] : 0.f, dh = a.dentropy ? a.dentropy[row] : 0.f,
              entropy = a.dentropy ? a.entropy[row] : 0.f;
  Pack<T, V> px[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int e0 = first + u * NT * V;
    if (e0 >= 0 && e0 + V <= a.V) {
      px[u] = ld_pack<T, V>(x + e0);
    } else {
#pragma unroll
      for (int c = 0; c < V; ++c)
        px[u].v[c] = (unsigned)(e0 + c) < (unsigned)a.V ? x[e0 + c] : narrow<T>(-INFINITY);
    }
  }
  const bool none = lse == -INFINITY;  // a row with nothing left has no gradient
  const float w = target >= 0 && target < a.V && !none ? dl : 0.f, h = none ? 0.f : dh;
  const bool careful = !(lse > (std::is_same<T, __half>::value ? -60000.f : -1e18f) && lse < 1e18f && fabsf(h) < 1e18f);
  const float2 l2 = make_float2(-lse, -lse);
  // w + h (d + entropy) = h d + c.
  const float2 h2 = make_float2(-h, -h), c2 = make_float2(-fmaf(h, entropy, w), -fmaf(h, entropy, w));
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int e0 = first + u * NT * V;
    float v[V];
    if (careful) {
      widen_pack(px[u], v);
      const float base = none ? 0.f : lse;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float lp = max_nan(v[c] - base, kLpFloor);
        v[c] = -lp_exp<T>(make_float2(lp, lp)).x * fmaf(h, lp + entropy, w);
      }
    } else {
      lp_grad_hold(px[u]);
      widen_pack(px[u], v);
      if constexpr (V == 1) {
        const float d = v[0] - lse;
        v[0] = lp_exp<T>(make_float2(d, d)).x * fmaf(h2.x, d, c2.x);
      } else {
#pragma unroll
        for (int c = 0; c < V; c += 2) {
          const float2 d = add2(make_float2(v[c], v[c + 1]), l2);
          const float2 g = mul2(lp_exp<T>(d), fma2(h2, d, c2));
          v[c] = g.x, v[c + 1] = g.y;
        }
      }
    }
    if ((unsigned long long)(target - e0) < (unsigned)V) {  // one pack of the row
#pragma unroll
      for (int c = 0; c < V; ++c) v[c] += e0 + c == target ? w : 0.f;
    }
    const Pack<T, V> out = narrow_pack<T, V>(v);
    if (e0 >= 0 && e0 + V <= a.V) {
      st_pack(dx + e0, out);
    } else {
#pragma unroll
      for (int c = 0; c < V; ++c)
        if ((unsigned)(e0 + c) < (unsigned)a.V) dx[e0 + c] = out.v[c];
    }
  }
}

// ---- launches ------------------------------------------------------------------------

template <class T> cudaError_t launch_logprob(const LogprobJob& j, const LaunchCtx& ctx) {
  LogprobArgs<T> a = {};
  a.logits = (const T*)j.logits;
  a.stride = j.stride;
  a.targets = j.targets;
  a.targets64 = j.targets64;
  a.logprob = j.logprob;
  a.entropy = j.entropy;
  a.lse = j.lse;
  a.top_values = j.top_values;
  a.top_ids = j.top_ids;
  a.V = (int)j.V;
  a.K = j.top;
  a.err = ctx.err;
  // A cluster shares a row while the rows alone leave SMs short of two CTAs each and each
  // CTA has a tile of its own.
  constexpr long long tile = (long long)kLpThreads * kLpPacks * (16 / sizeof(T));
  unsigned C = 1;
  while (C < (unsigned)kLpMaxCluster && j.N * C < 2ll * ctx.num_sms && C * tile < j.V) C *= 2;
  auto kernel = j.top ? logprob_kernel<T, true> : logprob_kernel<T, false>;
  constexpr int smem = kLpStages * kLpPacks * kLpThreads * 16;
  static_assert(smem + sizeof(LpShared) <= 55 * 1024, "four CTAs an SM");
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  profile_before(ctx);
  e = launch_pdl_cluster(kernel, (unsigned)(j.N * C), kLpThreads, C, smem, ctx.stream, a, C);
  profile_after(ctx);
  return e;
}

template <class T> cudaError_t launch_logprob_backward(const LogprobJob& j, const LaunchCtx& ctx) {
  constexpr int V = 16 / sizeof(T);
  LogprobGradArgs<T> a = {};
  a.logits = (const T*)j.logits;
  a.dlogits = (T*)j.dlogits;
  a.stride = j.stride;
  a.dstride = j.dstride;
  a.targets = j.targets;
  a.targets64 = j.targets64;
  a.lse = j.lse;
  a.entropy = j.entropy;
  a.dlogprob = j.dlogprob;
  a.dentropy = j.dentropy;
  a.V = (int)j.V;
  const bool wide = (uintptr_t)j.logits % 16 == (uintptr_t)j.dlogits % 16 &&
                    (j.N <= 1 || (j.stride - j.dstride) * (long long)sizeof(T) % 16 == 0);
  const long long per = (long long)kLpThreads * kLpGradPacks * (wide ? V : 1);
  a.blocks = (int)((j.V + (wide ? V - 1 : 0) + per - 1) / per);  // at the worst offset
  const long long grid = j.N * a.blocks;
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  profile_before(ctx);
  const cudaError_t e = wide ? launch_pdl(logprob_backward_kernel<T, V>, (unsigned)grid, kLpThreads, 0, ctx.stream, a)
                             : launch_pdl(logprob_backward_kernel<T, 1>, (unsigned)grid, kLpThreads, 0, ctx.stream, a);
  profile_after(ctx);
  return e;
}

}  // namespace gbs
