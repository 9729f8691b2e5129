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
// operations; fp64 adds run at a seventieth of fp32's rate), a warp's lanes are added in the same way,
// warps and CTAs in fp64.
//
// Reads one row of V where all drafts are accepted (or without the drafter's probabilities), else
// two.  Bound by the latency of its passes: a lane's next piece is not under way while it adds one.
// A request's row is cut among the CTAs of a cluster and their warps.  One pass finds the warps'
// sums; the CTAs exchange theirs through the cluster, and the one within whose slice the draw falls
// reads that warp's slice again: its warps an eighth each, and one warp the eighth.
//
// Measured (GB300, cold caches): 128 requests, 4 drafts of 128000 fp32 38 us, of which the kernel 30 (98.9 MB
// read: 0.49 of the copy rate; 0.33 instructions a cycle and scheduler); 4 requests of 50021 15.5 us.
#pragma once

#include "lm.cuh"
#include "lm.h"

namespace gbs {

constexpr int kVerifyWarps = 8, kVerifyThreads = 32 * kVerifyWarps;

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
  const T *p, *q;     // q: what is taken off (without a drafter's probabilities: not read)
  long long without;  // the token that is left out, or -1
};
// What a lane reads at once of p (and q): U packs of V values, `step` apart.
template <class T, int V, int U, bool Q> struct VerifyPiece {
  Pack<T, V> p[U], q[U];
  // Packs past `left` values from `at` are read as the pack at `at`, which exists.
  __device__ __forceinline__ void load(const VerifyRow<T>& r, long long at, int step, long long left) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long k = at + (u * step < left ? u * step : 0);
      p[u] = ld_pack<T, V>(r.p + k);
      if constexpr (Q) q[u] = ld_pack<T, V>(r.q + k);
    }
  }
  // What is left of pack u, and what the differences' roundings lost.  out: the place in the pack
  // of the token that is left out.
  __device__ __forceinline__ void rest(int u, bool there, long long out, float (&d)[V], float (&lost)[V]) const {
    float pv[V], qv[V];
    widen_pack(p[u], pv);
    if constexpr (Q) widen_pack(q[u], qv);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (!there || (!Q && e == out)) pv[e] = 0.f;
      if constexpr (Q) {
        d[e] = verify_rest(pv[e], fmaxf(qv[e], 0.f), lost[e]);
      } else {
        d[e] = pv[e] > 0.f ? pv[e] : 0.f;
        lost[e] = 0.f;
      }
    }
  }
};

// (lane 0's)
template <class T, int V, bool Q> __device__ double verify_sum(const VerifyRow<T>& r, long long s0, long long s1, int lane) {
  constexpr int U = V == 1 ? 12 : 16 / V;
  VerifySum sum;
  // A lane past the end of the slice reads its last pack, and counts it as nothing.
  for (long long from = s0; from < s1; from += 32 * V * U) {
    const long long left = s1 - from;
    const int own = lane * V;
    VerifyPiece<T, V, U, Q> piece;
    const auto add = [&](auto whole) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float d[V], lost[V];
        piece.rest(u, decltype(whole)::value || own + u * 32 * V < left, r.without - (from + own + u * 32 * V), d, lost);
#pragma unroll
        for (int e = 0; e < V; ++e) sum.add(d[e], lost[e]);
      }
    };
    if (left >= 32 * V * U) {
      piece.load(r, from + own, 32 * V, left);
      add(std::true_type());
    } else {
      piece.load(r, own < left ? from + own : s1 - V, 32 * V, left - own);
      add(std::false_type());
    }
  }
#pragma unroll
  for (int k = 16; k; k >>= 1) sum.add(__shfl_xor_sync(0xffffffffu, sum.hi, k), __shfl_xor_sync(0xffffffffu, sum.lo, k));
  return sum.value();
}

struct VerifyShared {
  double warp_sum[kVerifyWarps], cta_sum;
  double before, limit;  // of the draw: the sum before the slice, what has to be exceeded
  long long from, to;    // the slice; from < 0: not in this CTA
  int accepted;
};

static_assert(kVerifyWarps == 8 && kVerifyMaxCluster <= 8, "sums over 8 lanes");
// The sum of the lanes up to this one, of values of the first 8.
__device__ __forceinline__ double verify_scan8(double v, int lane) {
#pragma unroll
  for (int k = 1; k < 8; k <<= 1) {
    const double below = __shfl_up_sync(0xffffffffu, v, k);
    if (lane >= k) v += below;
  }
  return v;
}
// Of the lanes with something left, the first past the limit, or the last; -1: there is none.
__device__ __forceinline__ int verify_choose(bool some, bool past) {
  const unsigned all = __ballot_sync(0xffffffffu, some), over = __ballot_sync(0xffffffffu, some && past);
  return over ? __ffs(over) - 1 : all ? 31 - __clz(all) : -1;
}

// The first j in [from, to) with before + r_from + ... + r_j > limit; the last with r_j > 0 where
// rounding leaves none; -1 where no r_j is.  One warp, 8 neighbouring values a lane at a time.
template <class T, int V, bool Q>
__device__ long long verify_pick(const VerifyRow<T>& r, long long from, long long to, double before, double limit, int lane) {
  constexpr int E = 8, P = E / V;
  long long last = -1;
  for (; from < to; from += 32 * E) {
    const long long at = from + lane * E;
    VerifyPiece<T, V, P, Q> piece;
    piece.load(r, at < to ? at : from, V, to - at);
    const auto values = [&](auto&& each) {  // each(index, what is left, what its rounding lost), in order
#pragma unroll
      for (int u = 0; u < P; ++u) {
        float d[V], lost[V];
        piece.rest(u, at + u * V < to, r.without - (at + u * V), d, lost);
#pragma unroll
        for (int e = 0; e < V; ++e) each(u * V + e, d[e], lost[e]);
      }
    };
    VerifySum sum;
    int positive = -1;
    values([&](int e, float d, float lost) {
      sum.add(d, lost);
      if (d > 0.f) positive = e;
    });
    const double own = sum.value();
    double upto = own;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const double below = __shfl_up_sync(0xffffffffu, upto, k);
      if (lane >= k) upto += below;
    }
    const unsigned past = __ballot_sync(0xffffffffu, positive >= 0 && before + upto > limit);
    if (past) {
      const int first = __ffs(past) - 1;
      int j = -1;
      if (lane == first) {
        double s = before + (upto - own);
        values([&](int e, float d, float lost) {
          s += (double)d + (double)lost;
          if (j < 0 && d > 0.f && s > limit) j = e;
        });
        if (j < 0) j = positive;
      }
      return from + first * E + __shfl_sync(0xffffffffu, j, first);
    }
    const unsigned some = __ballot_sync(0xffffffffu, positive >= 0);
    if (some) last = from + (31 - __clz(some)) * E + __shfl_sync(0xffffffffu, positive, 31 - __clz(some));
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return last;
}

template <class T, int V>
__global__ void __launch_bounds__(kVerifyThreads, 4) verify_kernel(const __grid_constant__ VerifyArgs<T> a, unsigned C) {
  pdl_entry();
  __shared__ VerifyShared sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned rank = C > 1 ? cluster_rank() : 0;
  const long long b = blockIdx.x / C;

  // How many drafts are accepted (each CTA finds out for itself).  What is read for it is asked for
  // at once: the draft, then its probabilities.
  int length = a.lengths ? a.lengths[b] : a.K;
  float sample = 0.f;
  if (warp == 0) {
    sample = a.sample[b];
    bool bad = false;
    int n = a.K;
    for (int from = 0; from < a.K; from += 32) {
      const int i = from + lane;
      bool ok = i >= a.K;
      if (i < a.K) {
        const long long at = b * a.K + i;
        const float u = a.accept[at];
        const long long tok = a.tokens64 ? ((const long long*)a.tokens)[at] : ((const int*)a.tokens)[at];
        const bool real = tok >= 0 && tok < a.V;
        bad |= !real && i < length;
        if (real) {
          const float p = widen(a.target[b * a.tb + i * a.tt + tok]);
          const float q = a.draft ? fmaxf(widen(a.draft[b * a.qb + i * a.qt + tok]), 0.f) : 1.f;
          ok = (double)u * (double)q < (double)p;
        }
      }
      const unsigned no = __ballot_sync(0xffffffffu, !ok);
      if (no) {
        n = from + __ffs(no) - 1;
        break;
      }
      if (from + 32 >= length) break;
    }
    bad |= length < 0 || length > a.K;
    length = max(0, min(length, a.K));
    if (rank == 0 && bad) raise_err(a.err, ERRBIT_RANGE);
    if (lane == 0) sh.accepted = min(n, length);
  }
  length = max(0, min(length, a.K));
  __syncthreads();
  const int n = sh.accepted;
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
  double own = 0;
  if (s0 < s1) own = row.q ? verify_sum<T, V, true>(row, s0, s1, lane) : verify_sum<T, V, false>(row, s0, s1, lane);
  if (lane == 0) sh.warp_sum[warp] = own;
  __syncthreads();
  double slice = 0, slices = 0;
  if (warp == 0) {
    slice = lane < kVerifyWarps ? sh.warp_sum[lane] : 0.0;
    slices = verify_scan8(slice, lane);
    if (lane == kVerifyWarps - 1) sh.cta_sum = slices;
  }
  if (C > 1) cluster_sync();
  else __syncthreads();

  if (warp == 0) {  // where the draw falls: each CTA finds the same
    double mine = 0;
    if (lane < (int)C) mine = C > 1 ? from_u64<double>(ld_cluster_u64(cluster_addr(&sh.cta_sum, lane))) : sh.cta_sum;
    const double upto = verify_scan8(mine, lane), limit = (double)sample * __shfl_sync(0xffffffffu, upto, C - 1);
    const int owner = verify_choose(mine > 0, upto > limit);
    const double before = __shfl_sync(0xffffffffu, upto - mine, owner < 0 ? 0 : owner);
    const int k = verify_choose(slice > 0, before + slices > limit);
    const double skipped = __shfl_sync(0xffffffffu, slices - slice, k < 0 ? 0 : k);
    if (lane == 0) {
      const bool here = owner >= 0 && rank == (unsigned)owner && k >= 0;
      sh.from = here ? (long long)(rank * kVerifyWarps + k) * a.slice : -1;
      sh.to = min(a.V, sh.from + a.slice);
      sh.before = before + skipped;
      sh.limit = limit;
      if (owner < 0 && rank == 0) a.out[b * (a.K + 1) + n] = -1;
    }
  }
  __syncthreads();
  // The warps share that slice once more, and one of them picks the value.
  if (sh.from >= 0) {
    const long long sub = ((sh.to - sh.from + kVerifyWarps - 1) / kVerifyWarps + V - 1) / V * V;
    const long long f = sh.from + warp * sub, g = min(sh.to, f + sub);
    double part = 0;
    if (f < g) part = row.q ? verify_sum<T, V, true>(row, f, g, lane) : verify_sum<T, V, false>(row, f, g, lane);
    __syncthreads();  // the sums of the slices have been read
    if (lane == 0) sh.warp_sum[warp] = part;
    __syncthreads();
    if (warp == 0) {
      const double mine = lane < kVerifyWarps ? sh.warp_sum[lane] : 0.0, upto = verify_scan8(mine, lane);
      const int k = verify_choose(mine > 0, sh.before + upto > sh.limit);
      const double before = sh.before + __shfl_sync(0xffffffffu, upto - mine, k < 0 ? 0 : k);
      long long j = -1;
      if (k >= 0) {
        const long long from = sh.from + k * sub, to = min(sh.to, from + sub);
        j = row.q ? verify_pick<T, V, true>(row, from, to, before, sh.limit, lane)
                  : verify_pick<T, V, false>(row, from, to, before, sh.limit, lane);
      }
      if (lane == 0) a.out[b * (a.K + 1) + n] = (int32_t)j;
    }
  }
  if (rank == 0) {
    if (threadIdx.x == 0) a.accepted[b] = n;
    for (int i = threadIdx.x; i <= a.K; i += kVerifyThreads) {
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
  // CTAs of a request: as many as all fit at once, 4 an SM, while a warp has more than 512 values.
  unsigned C = 1;
  while (C < kVerifyMaxCluster && 2 * j.B * C <= 4 * ctx.num_sms && j.V > (long long)C * kVerifyWarps * 512) C *= 2;
  const long long step = 32 * V, warps = (long long)C * kVerifyWarps;
  a.slice = ((j.V + warps - 1) / warps + step - 1) / step * step;
  profile_before(ctx);
  const cudaError_t e =
      launch_pdl_cluster(verify_kernel<T, V>, (unsigned)(j.B * C), kVerifyThreads, C, 0, ctx.stream, a, C);
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
