// logprob.cuh -- log probabilities of given tokens from rows of logits, with the entropy
// of each row and its most likely alternatives, and the gradient.
//
//   lse = log sum exp(x_j),  logprob = x_target - lse,  p_j = exp(x_j - lse),
//   entropy = -sum p_j log p_j,  top: the K largest x_j in falling order, ties to the
//   lower index, with their log probabilities;
//   gradient:  dx_j = dlogprob ([j = target] - p_j) - dentropy p_j (log p_j + entropy).
//
// Each row is read once.  A thread keeps the running maximum m of its values and, relative
// to it, s = sum e^d and t = sum e^d d with d = x - m; when m grows by D, t becomes
// e^-D (t - s D) and s becomes e^-D s.  Then  lse = m + log s  and  entropy = log s - t/s,
// which loses nothing to cancellation.  A masked logit (-inf) has e^d = 0 and d is held at a
// finite floor, so that its product is 0 and not a NaN; a NaN or +inf logit
// makes the row's results NaN.
//
// The alternatives are found in the same pass, as a compaction: a value enters a buffer
// in shared memory if its key (the value in the high half, the index reversed in the low
// half: unique, so ties are settled) reaches a threshold that K values are known to reach.
// The first threshold is the K-th largest of 64 group maxima of the first tile, so a few
// dozen values pass of each tile; the buffer is sorted once at the end.  When it would
// overflow, it is sorted down to K, the threshold rises past the K-th, and what the tile
// could not place is offered again.
//
// With few rows a cluster of CTAs shares each row, slice by slice; CTA 0 of the cluster
// reads the others' sums and lists through distributed shared memory.
//
// Rows start anywhere: packs of 16 bytes are laid over the row from the boundary below its
// first value, and values outside the row or the slice count as masked.
#pragma once

#include <cfloat>

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
constexpr int kLpGroups = 64;      // groups of threads whose maxima give the first threshold
constexpr int kLpBuffer = 2048;    // keys
constexpr int kLpMaxCluster = 8;
// Differences from a maximum stop here: e^d has long been 0 in fp32, and products with
// d stay finite, so that 0 times them is 0.
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

// Running sums relative to the maximum.
struct LpSums {
  float m, s, t;
};
// Multiplies by e^(m_old - m_new) and moves t to the new maximum.
__device__ __forceinline__ void lp_rebase(LpSums& a, float m) {
  const float d = max_nan(a.m - m, kLpFloor), k = ex2(d * kLog2e);
  a.t = k * fmaf(a.s, d, a.t);
  a.s *= k;
  a.m = m;
}
__device__ __forceinline__ LpSums lp_join(LpSums a, LpSums b) {
  const float m = max_nan(a.m, b.m);
  lp_rebase(a, m);
  lp_rebase(b, m);
  return {m, a.s + b.s, a.t + b.t};
}

struct LpShared {
  unsigned long long keys[kLpBuffer];
  unsigned long long group[kLpGroups];
  LpSums warp[kLpThreads / 32];
  LpSums sums;  // the CTA's
  unsigned long long tau;
  int count;
};

// Sorts keys[0 .. n) in falling order (n is padded with zeros to a power of two).  All
// threads of the CTA call it, after a barrier; ends with a barrier.
__device__ __forceinline__ void lp_sort(unsigned long long* keys, int n) {
  int size = 32;
  while (size < n) size *= 2;
  for (int i = n + threadIdx.x; i < size; i += kLpThreads) keys[i] = 0;
  __syncthreads();
  for (int k = 2; k <= size; k *= 2) {
    for (int j = k / 2; j > 0; j /= 2) {
      for (int p = threadIdx.x; p < size / 2; p += kLpThreads) {
        const int i = 2 * p - (p & (j - 1)), q = i + j;
        const unsigned long long x = keys[i], y = keys[q];
        const bool falling = (i & k) == 0;
        if (falling ? x < y : x > y) {
          keys[i] = y;
          keys[q] = x;
        }
      }
      __syncthreads();
    }
  }
}

template <class T, bool TOP>
__global__ void __launch_bounds__(kLpThreads) logprob_kernel(const __grid_constant__ LogprobArgs<T> a, unsigned C) {
  constexpr int V = 16 / sizeof(T), U = kLpPacks, NT = kLpThreads;
  __shared__ LpShared sh;
  pdl_entry();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  if (TOP && tid == 0) {
    sh.count = 0;
    sh.tau = 0;
  }

  Pack<T, V> next[U];
  auto load = [&](int p) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = p + u * NT + tid;
      const int e0 = j * V - off;  // packs fit in 31 bits of values: V <= 2^31 - 1 - 16
      if (j < p1 && e0 >= 0 && e0 + V <= a.V) {
        next[u] = ld_pack<T, V>(x + e0);
      } else {
#pragma unroll
        for (int c = 0; c < V; ++c)
          next[u].v[c] = j < p1 && (unsigned)(e0 + c) < (unsigned)a.V ? x[e0 + c] : narrow<T>(-INFINITY);
      }
    }
  };
  LpSums sums = {-FLT_MAX, 0.f, 0.f};
  if (p0 < p1) load(p0);
  for (int p = p0; p < p1; p += U * NT) {
    float v[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) widen_pack(next[u], v[u]);
    if (p + U * NT < p1) load(p + U * NT);
    float best[U];  // the largest of each pack
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float g = v[u][0];
#pragma unroll
      for (int c = 1; c < V; ++c) g = max_nan(g, v[u][c]);
      best[u] = g;
      if (g > sums.m) lp_rebase(sums, g);
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float d = max_nan(v[u][c] - sums.m, kLpFloor), e = ex2(d * kLog2e);
        sums.s += e;
        sums.t = fmaf(e, d, sums.t);
      }
    }
    if constexpr (TOP) {
      auto index = [&](int u, int c) { return (p + u * NT + tid) * V - off + c; };
      auto inside = [&](int i) { return (unsigned)i < (unsigned)end; };
      // Raises the threshold to the K-th largest of 64 group maxima of this tile.
      auto tighten = [&]() {
        // This thread's largest value, at its first place inside the slice.
        float top = best[0];
#pragma unroll
        for (int u = 1; u < U; ++u) top = max_nan(top, best[u]);
        int at = -1;
#pragma unroll
        for (int u = U - 1; u >= 0; --u)
#pragma unroll
          for (int c = V - 1; c >= 0; --c)
            if ((v[u][c] == top || v[u][c] != v[u][c]) && inside(index(u, c))) at = index(u, c);
        unsigned long long k = at < 0 ? 0 : lp_key(top, at);
        constexpr int per_group = NT / kLpGroups;
#pragma unroll
        for (int d = 1; d < per_group; d *= 2) {
          const unsigned long long o = __shfl_xor_sync(0xffffffffu, k, d);
          k = o > k ? o : k;
        }
        if (tid % per_group == 0) sh.group[tid / per_group] = k;
        __syncthreads();
        // Each group's rank among the maxima, counted by its threads together.
        const unsigned long long mine = sh.group[tid / per_group];
        int above = 0;
        for (int g = tid % per_group; g < kLpGroups; g += per_group) above += sh.group[g] > mine;
#pragma unroll
        for (int d = 1; d < per_group; d *= 2) above += __shfl_xor_sync(0xffffffffu, above, d);
        if (tid % per_group == 0 && above == a.K - 1 && mine > sh.tau) sh.tau = mine;
        __syncthreads();
      };
      // Sorts the buffer down to the K largest and raises the threshold past the K-th.
      auto compress = [&]() {
        const int n = sh.count < kLpBuffer ? sh.count : kLpBuffer;
        __syncthreads();
        lp_sort(sh.keys, n);
        if (tid == 0) {
          sh.count = n < a.K ? n : a.K;
          if (n >= a.K && sh.keys[a.K - 1] + 1 > sh.tau) sh.tau = sh.keys[a.K - 1] + 1;
        }
        __syncthreads();
      };
      if (p == p0) {
        __syncthreads();  // count and tau are set
        tighten();
      }
      unsigned in = 0;  // which of this thread's values have entered the buffer
      static_assert(U * V <= 32, "one bit a value");
      for (;;) {
        const unsigned long long tau = sh.tau;
        const float bar = tau ? lp_unorder((unsigned)(tau >> 32)) : -INFINITY;
        bool full = false;
        // Few packs hold a value at or above the bar: theirs are read again (from L1 or
        // L2), which keeps this path's registers and code small.
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (best[u] < bar) continue;
#pragma unroll 1
          for (int c = 0; c < V; ++c) {
            const int i = index(u, c);
            if (!inside(i) || in >> (u * V + c) & 1) continue;
            const unsigned long long k = lp_key(widen(x[i]), i);
            if (k < tau) continue;
            const int at = atomicAdd(&sh.count, 1);
            if (at < kLpBuffer) {
              sh.keys[at] = k;
              in |= 1u << (u * V + c);
            } else {
              full = true;
            }
          }
        }
        // Each time round the buffer takes at least kLpBuffer - K more of the tile, so
        // this ends after a few rounds at most.
        if (!__syncthreads_or(full)) break;
        compress();
      }
    }
  }

  // The CTA's sums, in a fixed order.
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    LpSums o;
    o.m = __shfl_xor_sync(0xffffffffu, sums.m, d);
    o.s = __shfl_xor_sync(0xffffffffu, sums.s, d);
    o.t = __shfl_xor_sync(0xffffffffu, sums.t, d);
    sums = lp_join(sums, o);
  }
  if (lane == 0) sh.warp[warp] = sums;
  __syncthreads();
  if (tid == 0) {
    LpSums r = sh.warp[0];
    for (int w = 1; w < NT / 32; ++w) r = lp_join(r, sh.warp[w]);
    sh.sums = r;
  }
  if constexpr (TOP) {
    const int n = sh.count < kLpBuffer ? sh.count : kLpBuffer;
    lp_sort(sh.keys, n);  // begins and ends with a barrier
  }
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
        lp_sort(sh.keys, (int)C * a.K);
      }
    }
    cluster_sync();  // the others' shared memory has been read
  } else {
    __syncthreads();
  }
  if (rank != 0) return;
  const LpSums r = sh.sums;
  const float log_s = logf(r.s);
  if (tid == 0) {
    // A row with nothing left (all -inf) has s = 0: lse -inf, no entropy, logprob -inf.
    const bool none = r.s == 0.f;
    a.lse[row] = none ? -INFINITY : r.m + log_s;
    a.entropy[row] = none ? 0.f : log_s - r.t / r.s;
    a.logprob[row] = target < 0 ? 0.f : none ? -INFINITY : (xt - r.m) - log_s;
  }
  if constexpr (TOP) {
    if (tid < a.K) {
      const unsigned long long k = sh.keys[tid];
      a.top_ids[row * a.K + tid] = (int32_t)(0x7fffffffu - (unsigned)k);
      a.top_values[row * a.K + tid] = r.s == 0.f ? -INFINITY : (lp_unorder((unsigned)(k >> 32)) - r.m) - log_s;
    }
  }
}

// The gradient: one read and one write of each logit, U packs a thread.  Where the rows of
// the two arrays start at different offsets from a 16-byte boundary V is 1.
template <class T> struct LogprobGradArgs {
  const T* logits;
  T* dlogits;
  long long stride, dstride;
  const void* targets;
  int targets64;
  const float *lse, *entropy, *dlogprob, *dentropy;
  int V, blocks;  // blocks of a row
};

template <class T, int V>
__global__ void __launch_bounds__(kLpThreads) logprob_backward_kernel(const __grid_constant__ LogprobGradArgs<T> a) {
  constexpr int U = kLpPacks, NT = kLpThreads;
  pdl_entry();
  const long long row = blockIdx.x / a.blocks;
  const T* x = a.logits + row * a.stride;
  T* dx = a.dlogits + row * a.dstride;
  const int off = V == 1 ? 0 : (int)((uintptr_t)x % 16 / sizeof(T));
  const int p = (int)(blockIdx.x % a.blocks) * U * NT + threadIdx.x;
  Pack<T, V> px[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int e0 = (p + u * NT) * V - off;
    if (e0 >= 0 && e0 + V <= a.V) {
      px[u] = ld_pack<T, V>(x + e0);
    } else {
#pragma unroll
      for (int c = 0; c < V; ++c)
        px[u].v[c] = (unsigned)(e0 + c) < (unsigned)a.V ? x[e0 + c] : narrow<T>(-INFINITY);
    }
  }
  const long long target = lp_target(a.targets, a.targets64, row);
  const float lse = a.lse[row];
  const bool none = lse == -INFINITY;  // a row with nothing left has no gradient
  const float w = a.dlogprob && target >= 0 && target < a.V && !none ? a.dlogprob[row] : 0.f;
  const float h = a.dentropy && !none ? a.dentropy[row] : 0.f, entropy = a.dentropy ? a.entropy[row] : 0.f;
  const float base = none ? 0.f : lse;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int e0 = (p + u * NT) * V - off;
    float v[V];
    widen_pack(px[u], v);
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const float lp = max_nan(v[c] - base, kLpFloor);  // -inf: p = 0, and p lp = 0
      const float q = ex2(lp * kLog2e);
      v[c] = fmaf(-q, fmaf(h, lp + entropy, w), e0 + c == target ? w : 0.f);
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
  profile_before(ctx);
  const cudaError_t e = j.top ? launch_pdl_cluster(logprob_kernel<T, true>, (unsigned)(j.N * C), kLpThreads, C, 0,
                                                   ctx.stream, a, C)
                              : launch_pdl_cluster(logprob_kernel<T, false>, (unsigned)(j.N * C), kLpThreads, C, 0,
                                                   ctx.stream, a, C);
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
  const long long per = (long long)kLpThreads * kLpPacks * (wide ? V : 1);
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
