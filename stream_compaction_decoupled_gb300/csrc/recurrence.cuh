// recurrence.cuh -- the gated linear recurrence of a (batch, time, channel) array,
//   h_t = a_t h_{t-1} + u_t x_t,   a = sigmoid(f),   u = sigmoid(i) or 1 - a,
// its gradient, and its form for one token a call.
//
// Step t is the affine map y -> a_t y + b_t (b = u x), and maps compose associatively:
// (A1, B1) then (A2, B2) is (A1 A2, A2 B1 + B2).  A CTA owns W channels of one batch
// row for all of time and takes it tile by tile; the threads of a tile split its rows,
// each composes its own R rows, the threads' maps are composed across the warp and the
// CTA, and each thread then replays its rows from the state it starts from.  Every input
// is read once and every output written once, and the composition order is fixed, so a
// call's results do not vary from run to run.
//
// Where B*D/W CTAs would leave SMs idle, a cluster of C CTAs shares the strip: its CTAs
// take C consecutive tiles at a time and exchange their tiles' maps through distributed
// shared memory, one cluster barrier per round.  No CTA waits on another outside that
// hardware barrier, and no global scratch is needed.
//
// The gradient runs the same scan backwards in time.  With g_t = dL/dh_t (all paths) and
// c_t = a_t g_t,   g_t = dh_t + c_{t+1}   and   c_t = a_t c_{t+1} + a_t dh_t,
// which is again a map per row, of a_t and dh_t alone.  Then
//   dx_t = u_t g_t,   df_t = a_t (1 - a_t) h_{t-1} g_t,   di_t = u_t (1 - u_t) x_t g_t,
//   and without i:    df_t = a_t (1 - a_t) (h_{t-1} - x_t) g_t.
// Where starts[t] is set the state before t is dropped: a_t counts as 0 in the scan and
// h_{t-1} as 0 in df_t.
#pragma once

#include "lm.cuh"
#include "lm.h"

namespace gbs {

// sigmoid(z) and 1 - sigmoid(z) = sigmoid(-z), both to a few units in the last place at
// either end: e = exp(-z), 1/(1+e) and e/(1+e).  The exponent stops at 2^125, where the
// first is 0 to fp32 and the second still finite; a NaN stays a NaN.
__device__ __forceinline__ void sigmoid_both(float z, float& s, float& c) {
  const float e = ex2(min_nan(-z * kLog2e, 125.f));
  s = rcp(1.f + e);
  c = e * s;
}

template <class T> struct RecArgs {
  const T *x, *f, *i, *h, *dh;  // backward reads h and dh
  T *y, *dx, *df, *di;          // forward writes y
  long long xb, xt, fb, ft, ib, it, hb, ht, dhb, dht, yb, yt, dxb, dxt, dfb, dft, dib, dit;
  const float *h0, *dlast;
  const uint8_t* starts;
  float *last, *dh0;
  long long T_;
  int D, strips;  // strips of W channels per batch row
};

// Geometry.  V channels a thread (16 bytes, or 1 where rows are not 16-byte aligned),
// LANES threads of a warp side by side along the channels, the other lanes and the warps
// along time, R consecutive rows a thread.
template <int V_, int LANES_, int R_, int STAGES_> struct RecGeom {
  static constexpr int V = V_, LANES = LANES_, R = R_, STAGES = STAGES_;
  static constexpr int NT = 256, WARPS = NT / 32;
  static constexpr int W = V * LANES;
  static constexpr int GROUPS = 32 / LANES;
  static constexpr int L = WARPS * GROUPS * R;  // rows of a tile
};
constexpr int kRecMaxCluster = 8;

template <class G> struct RecShared {
  float a[G::WARPS][G::W], b[G::WARPS][G::W];  // the map of each warp's rows
  float from[G::WARPS][G::W];                  // the state each warp starts from
  float ca[2][G::W], cb[2][G::W];              // the CTA's map of this round and the last
};

// The state `in` that each thread's first row starts from, given the map (A, B) of its R
// rows and, in threads tid < W, the state `carry` before the cluster's rows of this
// round; updates `carry` to the state after them.  All threads call it.
template <class G>
__device__ __forceinline__ void rec_carry(float (&A)[G::V], float (&B)[G::V], float (&in)[G::V], RecShared<G>& sh,
                                          float& carry, unsigned C, unsigned rank, int round) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c0 = (lane % G::LANES) * G::V;
#pragma unroll
  for (int d = G::LANES; d < 32; d *= 2) {
#pragma unroll
    for (int k = 0; k < G::V; ++k) {
      const float pa = __shfl_up_sync(0xffffffffu, A[k], d), pb = __shfl_up_sync(0xffffffffu, B[k], d);
      if (lane >= d) {
        B[k] = fmaf(A[k], pb, B[k]);
        A[k] *= pa;
      }
    }
  }
  if (lane >= 32 - G::LANES) {
#pragma unroll
    for (int k = 0; k < G::V; ++k) {
      sh.a[warp][c0 + k] = A[k];
      sh.b[warp][c0 + k] = B[k];
    }
  }
  // From here on the map of the rows before this thread's in its warp.
#pragma unroll
  for (int k = 0; k < G::V; ++k) {
    if constexpr (G::GROUPS > 1) {
      const float pa = __shfl_up_sync(0xffffffffu, A[k], G::LANES), pb = __shfl_up_sync(0xffffffffu, B[k], G::LANES);
      A[k] = lane < G::LANES ? 1.f : pa;
      B[k] = lane < G::LANES ? 0.f : pb;
    } else {
      A[k] = 1.f;
      B[k] = 0.f;
    }
  }
  __syncthreads();
  float wa[G::WARPS], wb[G::WARPS];
  if (tid < G::W) {
#pragma unroll
    for (int w = 0; w < G::WARPS; ++w) {
      wa[w] = sh.a[w][tid];
      wb[w] = sh.b[w][tid];
    }
  }
  float start = carry;
  if (C > 1) {
    const int slot = round & 1;
    if (tid < G::W) {
      float ta = 1.f, tb = 0.f;
#pragma unroll
      for (int w = 0; w < G::WARPS; ++w) {
        tb = fmaf(wa[w], tb, wb[w]);
        ta *= wa[w];
      }
      sh.ca[slot][tid] = ta;
      sh.cb[slot][tid] = tb;
    }
    // Two slots in turn: a CTA writes a slot again only after the next round's barrier,
    // which every reader of the slot reaches after its reads.
    cluster_sync();
    if (tid < G::W) {
      float ra[kRecMaxCluster], rb[kRecMaxCluster];
#pragma unroll
      for (unsigned r = 0; r < kRecMaxCluster; ++r) {
        if (r < C) {
          ra[r] = ld_cluster_f32(cluster_addr(&sh.ca[slot][tid], r));
          rb[r] = ld_cluster_f32(cluster_addr(&sh.cb[slot][tid], r));
        }
      }
#pragma unroll
      for (unsigned r = 0; r < kRecMaxCluster; ++r) {
        if (r < C) {
          if (r == rank) start = carry;
          carry = fmaf(ra[r], carry, rb[r]);
        }
      }
    }
  }
  if (tid < G::W) {
    float s = start;
#pragma unroll
    for (int w = 0; w < G::WARPS; ++w) {
      sh.from[w][tid] = s;
      s = fmaf(wa[w], s, wb[w]);
    }
    if (C == 1) carry = s;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < G::V; ++k) in[k] = fmaf(A[k], sh.from[warp][c0 + k], B[k]);
}

// Where a thread's values of one array in one tile are: staged in shared memory by its
// own asynchronous copies (16-byte packs), or read straight from global memory.
template <class T, class G, int NA> struct RecStage {
  static constexpr size_t kSlot = (size_t)G::R * G::NT * 16;  // one array
  static constexpr size_t kStage = kSlot * NA;
  static constexpr size_t kBytes = G::V == 1 ? 0 : kStage * G::STAGES;
};

template <class T, bool GATE, class G>
__global__ void __launch_bounds__(G::NT) rec_forward_kernel(const __grid_constant__ RecArgs<T> a, unsigned C) {
  using S = RecStage<T, G, GATE ? 3 : 2>;
  constexpr int V = G::V, R = G::R;
  extern __shared__ __align__(16) unsigned char stage_mem[];
  __shared__ RecShared<G> sh;
  pdl_entry();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned rank = C > 1 ? cluster_rank() : 0;
  const unsigned strip = blockIdx.x / C;
  const long long b = strip / a.strips;
  const int d0 = (int)(strip % a.strips) * G::W;
  const int ch = d0 + (lane % G::LANES) * V;
  const bool live = ch < a.D;
  const int group = warp * G::GROUPS + lane / G::LANES;
  // The first row of this thread in its CTA's first tile.
  const long long row0 = (long long)rank * G::L + group * R;
  const long long step = (long long)C * G::L;
  const long long rounds = (a.T_ + step - 1) / step;
  const int chs = live ? ch : 0;  // an address that exists
  const T* x = a.x + b * a.xb + chs;
  const T* f = a.f + b * a.fb + chs;
  const T* g = GATE ? a.i + b * a.ib + chs : nullptr;
  T* y = a.y + b * a.yb + chs;
  const uint8_t* starts = a.starts ? a.starts + b * a.T_ : nullptr;

  float carry = 0.f;
  if (tid < G::W && d0 + tid < a.D && a.h0) carry = a.h0[b * a.D + d0 + tid];

  auto fetch = [&](long long k) {  // tile of round k into its stage
    if constexpr (V > 1) {
      unsigned char* base = stage_mem + (size_t)(k % G::STAGES) * S::kStage + (size_t)tid * 16;
      const long long t0 = row0 + k * step;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bool on = live && t0 + r < a.T_;
        const long long t = on ? t0 + r : 0;
        cp_async16(base + r * G::NT * 16, x + t * a.xt, on);
        cp_async16(base + S::kSlot + r * G::NT * 16, f + t * a.ft, on);
        if constexpr (GATE) cp_async16(base + 2 * S::kSlot + r * G::NT * 16, g + t * a.it, on);
      }
      cp_async_commit();
    }
  };
  if constexpr (V > 1) {
#pragma unroll
    for (int k = 0; k < G::STAGES - 1; ++k) {
      if (k < rounds) fetch(k);
      else cp_async_commit();
    }
  }
  for (long long k = 0; k < rounds; ++k) {
    const long long t0 = row0 + k * step;
    Pack<T, V> px[R], pf[R], pi[R];
    if constexpr (V == 1) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bool on = live && t0 + r < a.T_;
        const long long t = on ? t0 + r : 0;
        px[r].v[0] = on ? x[t * a.xt] : narrow<T>(0.f);
        pf[r].v[0] = on ? f[t * a.ft] : narrow<T>(0.f);
        if constexpr (GATE) pi[r].v[0] = on ? g[t * a.it] : narrow<T>(0.f);
      }
    }
    bool drop[R];
#pragma unroll
    for (int r = 0; r < R; ++r) drop[r] = starts && t0 + r < a.T_ && starts[t0 + r] != 0;
    if constexpr (V > 1) {
      if (k + G::STAGES - 1 < rounds) fetch(k + G::STAGES - 1);
      else cp_async_commit();
      cp_async_wait<G::STAGES - 1>();
      const unsigned char* base = stage_mem + (size_t)(k % G::STAGES) * S::kStage + (size_t)tid * 16;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        px[r] = ld_pack<T, V>((const T*)(base + r * G::NT * 16));
        pf[r] = ld_pack<T, V>((const T*)(base + S::kSlot + r * G::NT * 16));
        if constexpr (GATE) pi[r] = ld_pack<T, V>((const T*)(base + 2 * S::kSlot + r * G::NT * 16));
      }
    }
    float av[R][V], bv[R][V], A[V], B[V], in[V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float xs[V], fs[V], is[V];
      widen_pack(px[r], xs);
      widen_pack(pf[r], fs);
      if constexpr (GATE) widen_pack(pi[r], is);
#pragma unroll
      for (int c = 0; c < V; ++c) {
        float s, u;
        sigmoid_both(fs[c], s, u);
        if constexpr (GATE) {
          float unused;
          sigmoid_both(is[c], u, unused);
        }
        // Past the end the map is the identity, so that `carry` ends as the last state.
        const bool on = t0 + r < a.T_;
        av[r][c] = drop[r] ? 0.f : on ? s : 1.f;
        bv[r][c] = on ? u * xs[c] : 0.f;
        A[c] = r ? A[c] * av[r][c] : av[r][c];
        B[c] = r ? fmaf(av[r][c], B[c], bv[r][c]) : bv[r][c];
      }
    }
    rec_carry<G>(A, B, in, sh, carry, C, rank, (int)(k & 1));
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int c = 0; c < V; ++c) in[c] = fmaf(av[r][c], in[c], bv[r][c]);
      if (live && t0 + r < a.T_) st_pack(y + (t0 + r) * a.yt, narrow_pack<T, V>(in));
    }
  }
  if (a.last && rank == 0 && tid < G::W && d0 + tid < a.D) a.last[b * a.D + d0 + tid] = carry;
  if (C > 1) cluster_sync();  // no CTA leaves while another may read its shared memory
}

// Position p = 0, 1, ... counts rows from the end: t = T - 1 - p.
template <class T, bool GATE, class G>
__global__ void __launch_bounds__(G::NT) rec_backward_kernel(const __grid_constant__ RecArgs<T> a, unsigned C) {
  using S = RecStage<T, G, GATE ? 5 : 4>;
  constexpr int V = G::V, R = G::R;
  extern __shared__ __align__(16) unsigned char stage_mem[];
  __shared__ RecShared<G> sh;
  pdl_entry();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned rank = C > 1 ? cluster_rank() : 0;
  const unsigned strip = blockIdx.x / C;
  const long long b = strip / a.strips;
  const int d0 = (int)(strip % a.strips) * G::W;
  const int ch = d0 + (lane % G::LANES) * V;
  const bool live = ch < a.D;
  const int group = warp * G::GROUPS + lane / G::LANES;
  const long long row0 = (long long)rank * G::L + group * R;
  const long long step = (long long)C * G::L;
  const long long rounds = (a.T_ + step - 1) / step;
  const int chs = live ? ch : 0;
  const T* x = a.x + b * a.xb + chs;
  const T* f = a.f + b * a.fb + chs;
  const T* g = GATE ? a.i + b * a.ib + chs : nullptr;
  const T* h = a.h + b * a.hb + chs;
  const T* dh = a.dh + b * a.dhb + chs;
  const uint8_t* starts = a.starts ? a.starts + b * a.T_ : nullptr;

  float carry = 0.f;
  if (tid < G::W && d0 + tid < a.D && a.dlast) carry = a.dlast[b * a.D + d0 + tid];

  auto fetch = [&](long long k) {
    if constexpr (V > 1) {
      unsigned char* base = stage_mem + (size_t)(k % G::STAGES) * S::kStage + (size_t)tid * 16;
      const long long p0 = row0 + k * step;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bool on = live && p0 + r < a.T_;
        const long long t = on ? a.T_ - 1 - (p0 + r) : 0;
        unsigned char* q = base + r * G::NT * 16;
        cp_async16(q, f + t * a.ft, on);
        cp_async16(q + S::kSlot, dh + t * a.dht, on);
        cp_async16(q + 2 * S::kSlot, x + t * a.xt, on);
        cp_async16(q + 3 * S::kSlot, h + (t > 0 ? t - 1 : 0) * a.ht, on && t > 0);
        if constexpr (GATE) cp_async16(q + 4 * S::kSlot, g + t * a.it, on);
      }
      cp_async_commit();
    }
  };
  if constexpr (V > 1) {
#pragma unroll
    for (int k = 0; k < G::STAGES - 1; ++k) {
      if (k < rounds) fetch(k);
      else cp_async_commit();
    }
  }
  for (long long k = 0; k < rounds; ++k) {
    const long long p0 = row0 + k * step;
    const unsigned char* base = nullptr;
    Pack<T, V> px[R], pf[R], pi[R], ph[R], pd[R];
    if constexpr (V == 1) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bool on = live && p0 + r < a.T_;
        const long long t = on ? a.T_ - 1 - (p0 + r) : 0;
        const T zero = narrow<T>(0.f);
        pf[r].v[0] = on ? f[t * a.ft] : zero;
        pd[r].v[0] = on ? dh[t * a.dht] : zero;
        px[r].v[0] = on ? x[t * a.xt] : zero;
        ph[r].v[0] = on && t > 0 ? h[(t - 1) * a.ht] : zero;
        if constexpr (GATE) pi[r].v[0] = on ? g[t * a.it] : zero;
      }
    }
    bool drop[R];
#pragma unroll
    for (int r = 0; r < R; ++r) drop[r] = starts && p0 + r < a.T_ && starts[a.T_ - 1 - (p0 + r)] != 0;
    if constexpr (V > 1) {
      if (k + G::STAGES - 1 < rounds) fetch(k + G::STAGES - 1);
      else cp_async_commit();
      cp_async_wait<G::STAGES - 1>();
      base = stage_mem + (size_t)(k % G::STAGES) * S::kStage + (size_t)tid * 16;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        pf[r] = ld_pack<T, V>((const T*)(base + r * G::NT * 16));
        pd[r] = ld_pack<T, V>((const T*)(base + S::kSlot + r * G::NT * 16));
      }
    }
    float av[R][V], A[V], B[V], in[V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float fs[V], ds[V];
      widen_pack(pf[r], fs);
      widen_pack(pd[r], ds);
#pragma unroll
      for (int c = 0; c < V; ++c) {
        float s, u;
        sigmoid_both(fs[c], s, u);
        const bool on = p0 + r < a.T_;
        av[r][c] = drop[r] ? 0.f : on ? s : 1.f;
        const float bv = on ? av[r][c] * ds[c] : 0.f;
        A[c] = r ? A[c] * av[r][c] : av[r][c];
        B[c] = r ? fmaf(av[r][c], B[c], bv) : bv;
      }
    }
    rec_carry<G>(A, B, in, sh, carry, C, rank, (int)(k & 1));
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long t = a.T_ - 1 - (p0 + r);
      if (V > 1) {
        px[r] = ld_pack<T, V>((const T*)(base + 2 * S::kSlot + r * G::NT * 16));
        ph[r] = ld_pack<T, V>((const T*)(base + 3 * S::kSlot + r * G::NT * 16));
        if constexpr (GATE) pi[r] = ld_pack<T, V>((const T*)(base + 4 * S::kSlot + r * G::NT * 16));
      }
      float xs[V], fs[V], is[V], hs[V], ds[V], ox[V], of[V], oi[V];
      widen_pack(px[r], xs);
      widen_pack(pf[r], fs);
      widen_pack(ph[r], hs);
      widen_pack(pd[r], ds);
      if constexpr (GATE) widen_pack(pi[r], is);
      if (t == 0 && a.h0 && live) {
#pragma unroll
        for (int c = 0; c < V; ++c) hs[c] = a.h0[b * a.D + ch + c];
      }
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float gt = ds[c] + in[c];  // dL/dh_t
        float s, s1, u, u1;
        sigmoid_both(fs[c], s, s1);
        const float before = drop[r] ? 0.f : hs[c];
        if constexpr (GATE) {
          sigmoid_both(is[c], u, u1);
          of[c] = s * s1 * before * gt;
          oi[c] = u * u1 * xs[c] * gt;
          ox[c] = u * gt;
        } else {
          of[c] = s * s1 * (before - xs[c]) * gt;
          ox[c] = s1 * gt;
        }
        in[c] = av[r][c] * gt;
      }
      if (live && t >= 0) {
        st_pack(a.dx + b * a.dxb + ch + t * a.dxt, narrow_pack<T, V>(ox));
        st_pack(a.df + b * a.dfb + ch + t * a.dft, narrow_pack<T, V>(of));
        if constexpr (GATE) st_pack(a.di + b * a.dib + ch + t * a.dit, narrow_pack<T, V>(oi));
      }
    }
  }
  if (a.dh0 && rank == 0 && tid < G::W && d0 + tid < a.D) a.dh0[b * a.D + d0 + tid] = carry;
  if (C > 1) cluster_sync();
}

// One token: row b moves the state slots[b] of the pool on by one step, in place.  A
// negative slot is a padded row: its output is zero and no state moves.  Purely a read
// and a write of each value, one 16-byte pack a thread.
template <class T> struct RecStepArgs {
  const T *x, *f, *i;
  T* h;
  long long sx, sf, si, sh, pool;
  float* state;
  const int32_t* slots;
  int D, packs;  // packs of V channels in a row
  long long n;   // B * packs
  ErrSink err;
};

template <class T, bool GATE, int V>
__global__ void __launch_bounds__(128) rec_step_kernel(const __grid_constant__ RecStepArgs<T> a) {
  pdl_entry();
  const long long at = (long long)blockIdx.x * 128 + threadIdx.x;
  if (at >= a.n) return;
  const long long b = at / a.packs;
  const int ch = (int)(at % a.packs) * V;
  long long slot = a.slots ? (long long)a.slots[b] : b;
  if (slot >= a.pool) {  // no such state: reported, and the row treated as padding
    if (ch == 0) raise_err(a.err, ERRBIT_RANGE);
    slot = -1;
  }
  const Pack<T, V> px = ld_pack<T, V>(a.x + b * a.sx + ch);
  const Pack<T, V> pf = ld_pack<T, V>(a.f + b * a.sf + ch);
  Pack<T, V> pi;
  if constexpr (GATE) pi = ld_pack<T, V>(a.i + b * a.si + ch);
  float out[V];
#pragma unroll
  for (int c = 0; c < V; ++c) out[c] = 0.f;
  if (slot >= 0) {
    float* st = a.state + slot * a.D + ch;
    if constexpr (V == 1) {
      out[0] = st[0];
    } else {
#pragma unroll
      for (int c = 0; c < V; c += 4) {
        const float4 q = *(const float4*)(st + c);
        out[c] = q.x, out[c + 1] = q.y, out[c + 2] = q.z, out[c + 3] = q.w;
      }
    }
    float xs[V], fs[V], is[V];
    widen_pack(px, xs);
    widen_pack(pf, fs);
    if constexpr (GATE) widen_pack(pi, is);
#pragma unroll
    for (int c = 0; c < V; ++c) {
      float s, u;
      sigmoid_both(fs[c], s, u);
      if constexpr (GATE) {
        float unused;
        sigmoid_both(is[c], u, unused);
      }
      out[c] = fmaf(s, out[c], u * xs[c]);
    }
    if constexpr (V == 1) {
      st[0] = out[0];
    } else {
#pragma unroll
      for (int c = 0; c < V; c += 4) *(float4*)(st + c) = make_float4(out[c], out[c + 1], out[c + 2], out[c + 3]);
    }
  }
  st_pack(a.h + b * a.sh + ch, narrow_pack<T, V>(out));
}

// ---- launches ------------------------------------------------------------------------

// Whether every row of the array starts on a 16-byte boundary.
template <class T> bool rows16(const SeqArray& s, long long B, long long T_) {
  if (!s.p) return true;
  return (uintptr_t)s.p % 16 == 0 && (B <= 1 || s.sb * (long long)sizeof(T) % 16 == 0) &&
         (T_ <= 1 || s.st * (long long)sizeof(T) % 16 == 0);
}

template <class T> RecArgs<T> rec_args(const RecurrenceJob& j) {
  RecArgs<T> a = {};
  a.x = (const T*)j.x.p, a.xb = j.x.sb, a.xt = j.x.st;
  a.f = (const T*)j.f.p, a.fb = j.f.sb, a.ft = j.f.st;
  a.i = (const T*)j.i.p, a.ib = j.i.sb, a.it = j.i.st;
  a.h = (const T*)j.h.p, a.hb = j.h.sb, a.ht = j.h.st;
  a.y = (T*)j.h.p, a.yb = j.h.sb, a.yt = j.h.st;
  a.dh = (const T*)j.dh.p, a.dhb = j.dh.sb, a.dht = j.dh.st;
  a.dx = (T*)j.dx.p, a.dxb = j.dx.sb, a.dxt = j.dx.st;
  a.df = (T*)j.df.p, a.dfb = j.df.sb, a.dft = j.df.st;
  a.di = (T*)j.di.p, a.dib = j.di.sb, a.dit = j.di.st;
  a.h0 = j.h0, a.dlast = j.dlast, a.starts = j.starts, a.last = j.last, a.dh0 = j.dh0;
  a.T_ = j.T, a.D = (int)j.D;
  return a;
}

// CTAs per cluster: doubled while the strips alone leave SMs short of two CTAs each and
// there are tiles to share.
template <class G> unsigned rec_cluster(long long strips, long long T_, int num_sms) {
  unsigned c = 1;
  while (c < (unsigned)kRecMaxCluster && strips * c < 2ll * num_sms && (long long)c * G::L < T_) c *= 2;
  return c;
}

template <class T, class G, int NA, class K>
cudaError_t rec_launch(K kernel, const RecurrenceJob& j, RecArgs<T> a, const LaunchCtx& ctx) {
  const long long strips = (j.D + G::W - 1) / G::W;
  const unsigned C = rec_cluster<G>(strips * j.B, j.T, ctx.num_sms);
  a.strips = (int)strips;
  const size_t smem = RecStage<T, G, NA>::kBytes;
  cudaError_t e = cudaSuccess;
  if (smem) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  profile_before(ctx);
  e = launch_pdl_cluster(kernel, (unsigned)(strips * j.B * C), G::NT, C, smem, ctx.stream, a, C);
  profile_after(ctx);
  return e;
}

template <class T> cudaError_t launch_recurrence(const RecurrenceJob& j, const LaunchCtx& ctx) {
  constexpr int V = 16 / sizeof(T);
  using GV = RecGeom<V, 8, 4, 2>;
  using GS = RecGeom<1, 32, 8, 1>;
  const RecArgs<T> a = rec_args<T>(j);
  const bool wide = j.D % V == 0 && rows16<T>(j.x, j.B, j.T) && rows16<T>(j.f, j.B, j.T) &&
                    rows16<T>(j.i, j.B, j.T) && rows16<T>(j.h, j.B, j.T);
  if (j.i.p)
    return wide ? rec_launch<T, GV, 3>(rec_forward_kernel<T, true, GV>, j, a, ctx)
                : rec_launch<T, GS, 3>(rec_forward_kernel<T, true, GS>, j, a, ctx);
  return wide ? rec_launch<T, GV, 2>(rec_forward_kernel<T, false, GV>, j, a, ctx)
              : rec_launch<T, GS, 2>(rec_forward_kernel<T, false, GS>, j, a, ctx);
}

template <class T> cudaError_t launch_recurrence_backward(const RecurrenceJob& j, const LaunchCtx& ctx) {
  constexpr int V = 16 / sizeof(T);
  using GV = RecGeom<V, 8, 2, 2>;
  using GS = RecGeom<1, 32, 4, 1>;
  const RecArgs<T> a = rec_args<T>(j);
  bool wide = j.D % V == 0;
  for (const SeqArray* s : {&j.x, &j.f, &j.i, &j.h, &j.dh, &j.dx, &j.df, &j.di}) wide = wide && rows16<T>(*s, j.B, j.T);
  if (j.i.p)
    return wide ? rec_launch<T, GV, 5>(rec_backward_kernel<T, true, GV>, j, a, ctx)
                : rec_launch<T, GS, 5>(rec_backward_kernel<T, true, GS>, j, a, ctx);
  return wide ? rec_launch<T, GV, 4>(rec_backward_kernel<T, false, GV>, j, a, ctx)
              : rec_launch<T, GS, 4>(rec_backward_kernel<T, false, GS>, j, a, ctx);
}

template <class T, bool GATE, int V>
cudaError_t rec_step(const RecurrenceStepJob& j, const LaunchCtx& ctx) {
  RecStepArgs<T> a = {};
  a.x = (const T*)j.x, a.f = (const T*)j.f, a.i = (const T*)j.i, a.h = (T*)j.h;
  a.sx = j.sx, a.sf = j.sf, a.si = j.si, a.sh = j.sh;
  a.pool = j.pool, a.state = j.state, a.slots = j.slots, a.D = (int)j.D;
  a.packs = (int)(j.D / V);
  a.n = j.B * a.packs;
  a.err = ctx.err;
  profile_before(ctx);
  const cudaError_t e =
      launch_pdl(rec_step_kernel<T, GATE, V>, (unsigned)((a.n + 127) / 128), 128, 0, ctx.stream, a);
  profile_after(ctx);
  return e;
}

template <class T> cudaError_t launch_recurrence_step(const RecurrenceStepJob& j, const LaunchCtx& ctx) {
  constexpr int V = 16 / sizeof(T);
  auto ok = [&](const void* p, long long s) {
    return !p || ((uintptr_t)p % 16 == 0 && (j.B <= 1 || s * (long long)sizeof(T) % 16 == 0));
  };
  const bool wide = j.D % V == 0 && ok(j.x, j.sx) && ok(j.f, j.sf) && ok(j.i, j.si) && ok(j.h, j.sh) &&
                    (uintptr_t)j.state % 16 == 0;  // a state row is D floats: a multiple of 16 bytes with D % V == 0
  if (j.i) return wide ? rec_step<T, true, V>(j, ctx) : rec_step<T, true, 1>(j, ctx);
  return wide ? rec_step<T, false, V>(j, ctx) : rec_step<T, false, 1>(j, ctx);
}

}  // namespace gbs
