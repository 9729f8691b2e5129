// verify_drafts.cuh -- which drafted tokens the target's probabilities accept, and the token
// that follows them, from given random numbers.
//
// Draft i of a request (token d, target probability p_i(d), drafter's q_i(d), or 1 without the
// drafter's probabilities) is accepted while  accept_i q_i(d) < p_i(d).  At the first that is not,
// n, the token is drawn from the rest  r_j = max(p_n(j) - q_n(j), 0)  (without the drafter's:
// p_n but for d); after all of them, from r = p_n of the row behind the last draft.  Drawn: the
// smallest j with  r_0 + ... + r_j > sample (r_0 + ... + r_{V-1}).
//
// A whole number is the result, so the sums are as good as exact: with an fp32 sum's errors one
// draw in a few dozen over a flat row of 128000 would fall on the wrong side of a border.  Each
// lane adds with the rounding errors kept (an error-free difference p - q and sum, ten fp32
// operations; fp64 adds run at a sixty-fourth of fp32's rate), lanes and warps in fp64.
//
// Bound by memory: one or two rows of V.  A request's row is cut among the CTAs of a cluster and
// their warps.  One pass finds the warps' sums; the CTAs exchange theirs through the cluster, and
// the one warp within whose slice the draw falls reads it again, some thousand values.
#pragma once

#include "lm.cuh"
#include "lm.h"

namespace gbs {

constexpr int kVerifyWarps = 16;

template <class T> struct VerifyArgs {
  const T *target, *draft;
  long long tb, tt, qb, qt;
  const void* tokens;
  const float *accept, *sample;
  const int32_t* lengths;
  int32_t *accepted, *out;
  long long V, slice;  // values of a warp, a multiple of what it reads at once
  int K, tokens64;
  ErrSink err;
};

// A sum with what its roundings lost.
struct VerifySum {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float v, float lost) {
    const float s = __fadd_rn(hi, v), b = __fsub_rn(s, hi);
    const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(v, b));
    hi = s;
    lo = __fadd_rn(lo, __fadd_rn(e, lost));
  }
  __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
};
// max(p - q, 0) (0 where p is NaN) and what its rounding lost: p > q >= 0, so the loss is exact.
__device__ __forceinline__ float verify_rest(float p, float q, float& lost) {
  const bool more = p > q;
  const float d = more ? __fsub_rn(p, q) : 0.f;
  lost = more ? __fsub_rn(__fsub_rn(p, d), q) : 0.f;
  return d;
}

// The rows that a request's draw is made from.
template <class T> struct VerifyRow {
  const T *p, *q;    // q null: nothing is taken off
  long long without;  // the token that is left out, or -1
  template <int V> __device__ __forceinline__ void load(long long at, long long end, float (&pv)[V], float (&qv)[V]) const {
    if (at < end) {
      widen_pack(ld_pack<T, V>(p + at), pv);
      if (q) widen_pack(ld_pack<T, V>(q + at), qv);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (at >= end) pv[e] = 0.f;
      if (at >= end || !q) qv[e] = 0.f;
      if (at + e == without) pv[e] = 0.f;
      qv[e] = fmaxf(qv[e], 0.f);
    }
  }
};

template <class T, int V> __device__ double verify_sum(const VerifyRow<T>& r, long long s0, long long s1, int lane) {
  constexpr int U = 4;
  VerifySum sum;
  for (long long at = s0 + lane * V; at < s1; at += 32 * V * U) {
    float p[U][V], q[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) r.load(at + u * 32 * V, s1, p[u], q[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float lost;
        const float d = verify_rest(p[u][e], q[u][e], lost);
        sum.add(d, lost);
      }
    }
  }
  double s = sum.value();
#pragma unroll
  for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
  return s;
}

// The first j of the slice with before + r_s0 + ... + r_j > limit; the last with r_j > 0 where
// rounding leaves none; -1 where no r_j is.
template <class T, int V>
__device__ long long verify_pick(const VerifyRow<T>& r, long long s0, long long s1, int lane, double before, double limit) {
  long long last = -1;
  for (long long from = s0; from < s1; from += 32 * V) {
    const long long at = from + lane * V;
    float p[V], q[V], d[V], lost[V];
    r.load(at, s1, p, q);
    double own = 0;
    long long positive = -1;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      d[e] = verify_rest(p[e], q[e], lost[e]);
      own += (double)d[e] + (double)lost[e];
      if (d[e] > 0.f) positive = at + e;
    }
    double upto = own;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const double below = __shfl_up_sync(0xffffffffu, upto, k);
      if (lane >= k) upto += below;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + upto > limit && positive >= 0);
    if (past) {
      const int first = __ffs(past) - 1;
      long long j = -1;
      if (lane == first) {
        double s = before + (upto - own);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          s += (double)d[e] + (double)lost[e];
          if (j < 0 && d[e] > 0.f && s > limit) j = at + e;
        }
        if (j < 0) j = positive;
      }
      return __shfl_sync(0xffffffffu, j, first);
    }
    const unsigned some = __ballot_sync(0xffffffffu, positive >= 0);
    if (some) last = __shfl_sync(0xffffffffu, positive, 31 - __clz(some));
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return last;
}

template <class T, int V>
__global__ void __launch_bounds__(kVerifyWarps * 32) verify_kernel(const __grid_constant__ VerifyArgs<T> a, unsigned C) {
  pdl_entry();
  __shared__ double warp_sum[kVerifyWarps];
  __shared__ double cta_sum;
  __shared__ int drafts_accepted;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned rank = C > 1 ? cluster_rank() : 0;
  const long long b = blockIdx.x / C;

  // How many drafts are accepted (each CTA finds out for itself).
  int length = a.lengths ? a.lengths[b] : a.K;
  const bool wrong = length < 0 || length > a.K;
  length = max(0, min(length, a.K));
  if (warp == 0) {
    bool bad = wrong;
    int n = length;
    for (int from = 0; from < length; from += 32) {
      const int i = from + lane;
      bool ok = true;
      if (i < length) {
        const long long at = b * a.K + i;
        const long long tok = a.tokens64 ? ((const long long*)a.tokens)[at] : ((const int*)a.tokens)[at];
        ok = tok >= 0 && tok < a.V;
        bad |= !ok;
        if (ok) {
          const float p = widen(a.target[b * a.tb + i * a.tt + tok]);
          const float q = a.draft ? fmaxf(widen(a.draft[b * a.qb + i * a.qt + tok]), 0.f) : 1.f;
          ok = (double)a.accept[at] * (double)q < (double)p;
        }
      }
      const unsigned no = __ballot_sync(0xffffffffu, !ok);
      if (no) {
        n = from + __ffs(no) - 1;
        break;
      }
    }
    if (rank == 0 && bad) raise_err(a.err, ERRBIT_RANGE);
    if (lane == 0) drafts_accepted = n;
  }
  __syncthreads();
  const int n = drafts_accepted;
  VerifyRow<T> row = {a.target + b * a.tb + n * a.tt, nullptr, -1};
  if (n < length) {
    if (a.draft) {
      row.q = a.draft + b * a.qb + n * a.qt;
    } else {
      const long long at = b * a.K + n;
      row.without = a.tokens64 ? ((const long long*)a.tokens)[at] : ((const int*)a.tokens)[at];
    }
  }

  const long long s0 = (long long)(rank * kVerifyWarps + warp) * a.slice, s1 = min(a.V, s0 + a.slice);
  const double own = s0 < s1 ? verify_sum<T, V>(row, s0, s1, lane) : 0.0;
  if (lane == 0) warp_sum[warp] = own;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0;
#pragma unroll
    for (int w = 0; w < kVerifyWarps; ++w) s += warp_sum[w];
    cta_sum = s;
  }
  if (C > 1) cluster_sync();
  else __syncthreads();

  if (warp == 0) {
    double total = 0, before = 0;
    unsigned owner = C, positive = C;
    double sums[kVerifyMaxCluster];
    for (unsigned c = 0; c < C; ++c) {
      const double s = C > 1 ? from_u64<double>(ld_cluster_u64(cluster_addr(&cta_sum, c))) : cta_sum;
      sums[c] = s;
      total += s;
      if (s > 0) positive = c;
    }
    const double limit = (double)a.sample[b] * total;
    double upto = 0;
    for (unsigned c = 0; c < C; ++c) {
      const double next = upto + sums[c];
      if (owner == C && sums[c] > 0 && next > limit) owner = c, before = upto;
      if (owner == C && c == positive) before = upto;
      upto = next;
    }
    if (owner == C) owner = positive;
    if (rank == (owner == C ? 0 : owner)) {
      long long j = -1;
      if (owner < C) {
        int w = -1, some = -1;
        double s = before, at = before, at_some = before;
        for (int k = 0; k < kVerifyWarps; ++k) {
          const double next = s + warp_sum[k];
          if (w < 0 && warp_sum[k] > 0) {
            some = k, at_some = s;
            if (next > limit) w = k, at = s;
          }
          s = next;
        }
        if (w < 0) w = some, at = at_some;
        if (w >= 0) {
          const long long f = (long long)(rank * kVerifyWarps + w) * a.slice;
          j = verify_pick<T, V>(row, f, min(a.V, f + a.slice), lane, at, limit);
        }
      }
      if (lane == 0) a.out[b * (a.K + 1) + n] = (int32_t)j;
    }
  }
  if (rank == 0) {
    if (threadIdx.x == 0) a.accepted[b] = n;
    for (int i = threadIdx.x; i <= a.K; i += kVerifyWarps * 32) {
      const long long at = b * a.K + i;
      if (i < n) a.out[b * (a.K + 1) + i] = a.tokens64 ? (int32_t)((const long long*)a.tokens)[at] : ((const int32_t*)a.tokens)[at];
      else if (i > n) a.out[b * (a.K + 1) + i] = -1;
    }
  }
  if (C > 1) cluster_sync_relaxed();  // no CTA leaves while another may still read its sum
}

template <class T, int V> cudaError_t verify_launch(const VerifyJob& j, const LaunchCtx& ctx) {
  VerifyArgs<T> a = {};
  a.target = (const T*)j.target, a.tb = j.tb, a.tt = j.tt;
  a.draft = (const T*)j.draft, a.qb = j.qb, a.qt = j.qt;
  a.tokens = j.tokens, a.tokens64 = j.tokens64, a.accept = j.accept, a.sample = j.sample, a.lengths = j.lengths;
  a.accepted = j.accepted, a.out = j.out, a.V = j.V, a.K = (int)j.K;
  a.err = ctx.err;
  // CTAs of a request: while there are fewer than two an SM and a warp has more than 512 values.
  unsigned C = 1;
  while (C < kVerifyMaxCluster && j.B * C < 2 * ctx.num_sms && j.V > (long long)C * kVerifyWarps * 512) C *= 2;
  const long long step = 32 * V, warps = (long long)C * kVerifyWarps;
  a.slice = ((j.V + warps - 1) / warps + step - 1) / step * step;
  profile_before(ctx);
  const cudaError_t e =
      launch_pdl_cluster(verify_kernel<T, V>, (unsigned)(j.B * C), kVerifyWarps * 32, C, 0, ctx.stream, a, C);
  profile_after(ctx);
  return e;
}

template <class T> cudaError_t launch_verify(const VerifyJob& j, const LaunchCtx& ctx) {
  constexpr int V = 16 / sizeof(T);
  const auto ok = [&](const void* p, long long sb, long long st, long long rows) {
    return !p || ((uintptr_t)p % 16 == 0 && (j.B <= 1 || sb % V == 0) && (rows <= 1 || st % V == 0));
  };
  const bool wide = j.V % V == 0 && ok(j.target, j.tb, j.tt, j.K + 1) && ok(j.draft, j.qb, j.qt, j.K);
  return wide ? verify_launch<T, V>(j, ctx) : verify_launch<T, 1>(j, ctx);
}

}  // namespace gbs
