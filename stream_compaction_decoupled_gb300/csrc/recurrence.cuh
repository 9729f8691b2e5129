// recurrence.cuh -- the gated linear recurrence of a (batch, time, channel) array,
//   h_t = a_t h_{t-1} + u_t x_t,   a = sigmoid(f),   u = sigmoid(i) or 1 - a,
// its gradient, and its form for one token a call.
//
// Step t is the affine map y -> a_t y + b_t (b = u x), and maps compose associatively:
// (A1, B1) then (A2, B2) is (A1 A2, A2 B1 + B2).  A CTA owns 64 channels of one batch row
// for all of time and takes them tile by tile.  The 8 warps of a tile split its rows, a
// lane holds 2 channels: each thread composes the maps of its R rows, the warps' maps meet
// in shared memory, and each thread replays its rows from the state they start from.  Every
// input is read once and every output written once, and the composition order is fixed, so
// results do not vary from run to run.
//
// Tiles reach shared memory by asynchronous copies of 16 bytes, STAGES - 1 tiles ahead of
// the one in hand.  Rows may start anywhere: where they are not all on 16-byte boundaries
// (EDGE) the copies start at the boundary below each row's first channel and each lane
// picks its channels out at the row's offset; a copy never reads outside its row.
//
// Where B*D/64 CTAs would leave SMs idle, a cluster of C CTAs shares the strip: its CTAs
// take C consecutive tiles at a time and send each other their tiles' maps through
// distributed shared memory, one cluster barrier per round.  No CTA waits on another
// outside that hardware barrier, and no global scratch is needed.
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

// sigmoid(z) alone: 1 / (1 + exp(-z)); exp(-z) may overflow to infinity, which gives 0.
__device__ __forceinline__ float sigmoid(float z) { return rcp(1.f + ex2(-z * kLog2e)); }

constexpr int kRecMaxCluster = 8;

// R rows a thread, so that a tile of one array is 8 KB whatever the type.
template <class T, bool EDGE_, int STAGES_> struct RecGeom {
  static constexpr bool EDGE = EDGE_;
  static constexpr int STAGES = STAGES_;
  static constexpr int NT = 256, WARPS = NT / 32, W = 64;
  static constexpr int V = 16 / sizeof(T);
  static constexpr int R = 16 / sizeof(T);
  static constexpr int L = WARPS * R;                        // rows of a tile
  static constexpr int CHUNKS = W / V + (EDGE ? 1 : 0);      // 16-byte copies of a row
  static constexpr int PITCH = CHUNKS * 16;                  // bytes of a row in shared memory
  static constexpr int ARRAY = L * PITCH;
  static constexpr int ITERS = (L * CHUNKS + NT - 1) / NT;   // copies of a thread for one array
};

// The maps of two channels.
struct RecShared {
  float4 warp[2][8][32];                  // (A, B) of each warp's rows, by lane; two rounds in turn
  float4 cta[2][kRecMaxCluster][32];      // of each CTA's tile
};

// One array of one strip: `p` is (b, t = 0, d0).
template <class T> struct RecStrip {
  const T* p;
  long long st;
};

// Copies row `t` of the strip, or nothing where `on` is false, into row `r` of its tile:
// this thread's share, chunk c.
template <class T, class G>
__device__ __forceinline__ void rec_copy(unsigned char* tile, const RecStrip<T>& s, int r, int c, long long t, bool on,
                                         int d0, int D) {
  unsigned char* dst = tile + r * G::PITCH + c * 16;
  const T* row = s.p + (on ? t : 0) * s.st;
  if constexpr (!G::EDGE) {
    const bool live = on && d0 + c * G::V < D;
    cp_async16(dst, live ? row + c * G::V : s.p, live);
  } else {
    const int off = (int)((uintptr_t)row % 16 / sizeof(T));
    const int e = c * G::V - off, ch = d0 + e;  // the chunk's first channel
    if (!on || e >= G::W || ch >= D) return;    // none of it is used
    if (ch >= 0) {
      const int n = D - ch < G::V ? D - ch : G::V;
      cp_async_part(dst, row + e, n * (int)sizeof(T));
    } else {  // the row begins inside the chunk
      for (int k = -ch; k < G::V && ch + k < D; ++k) ((T*)dst)[k] = row[e + k];
    }
  }
}

// The two channels of this lane in row `r` of a tile, which holds row `t` of the strip.
template <class T, class G>
__device__ __forceinline__ float2 rec_pair(const unsigned char* tile, const RecStrip<T>& s, int r, int lane, long long t) {
  const unsigned char* row = tile + r * G::PITCH;
  if constexpr (!G::EDGE) {
    if constexpr (sizeof(T) == 4) {
      return *(const float2*)(row + lane * 8);
    } else {
      Pair<T> q;
      const unsigned u = *(const unsigned*)(row + lane * 4);
      memcpy(&q, &u, 4);
      return make_float2(widen(q.x), widen(q.y));
    }
  } else {
    const unsigned off = (unsigned)((uintptr_t)(s.p + t * s.st) % 16);
    const T* q = (const T*)(row + off) + 2 * lane;
    return make_float2(widen(q[0]), widen(q[1]));
  }
}

// Writes the two channels ch, ch + 1 of a row; `p` points at the first.
template <class T, bool EDGE> __device__ __forceinline__ void rec_store(T* p, float2 v, int ch, int D) {
  if constexpr (!EDGE) {
    if (ch < D) {
      if constexpr (sizeof(T) == 4) {
        *(float2*)p = v;
      } else {
        const Pair<T> q = {narrow<T>(v.x), narrow<T>(v.y)};
        unsigned u;
        memcpy(&u, &q, 4);
        *(unsigned*)p = u;
      }
    }
  } else {
    if (ch < D) p[0] = narrow<T>(v.x);
    if (ch + 1 < D) p[1] = narrow<T>(v.y);
  }
}

// The states (two channels) that this warp's first row starts from, given the map m of its
// rows and the states `carry` before the cluster's rows of this round; moves `carry` past
// them.  All threads of the CTA call it.
__device__ __forceinline__ float2 rec_exchange(float4 m, float2& carry, RecShared& sh, unsigned C, unsigned rank,
                                               int turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  sh.warp[turn][warp][lane] = m;
  __syncthreads();
  if (C == 1) {
    float2 s = carry, in = carry;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const float4 q = sh.warp[turn][w][lane];
      if (w == warp) in = s;
      s = make_float2(fmaf(q.x, s.x, q.y), fmaf(q.z, s.y, q.w));
    }
    carry = s;
    return in;
  }
  float4 all = make_float4(1.f, 0.f, 1.f, 0.f), before = all;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const float4 q = sh.warp[turn][w][lane];
    if (w == warp) before = all;
    all = make_float4(all.x * q.x, fmaf(q.x, all.y, q.y), all.z * q.z, fmaf(q.z, all.w, q.w));
  }
  // Warp r sends the CTA's map to CTA r.  A CTA writes a slot again two rounds later, past
  // a barrier that its reader reaches after reading it.
  if ((unsigned)warp < C) st_cluster_f4(cluster_addr(&sh.cta[turn][rank][lane], (unsigned)warp), all);
  cluster_sync();
  float2 s = carry, start = carry;
#pragma unroll
  for (unsigned r = 0; r < kRecMaxCluster; ++r) {
    if (r < C) {
      const float4 q = sh.cta[turn][r][lane];
      if (r == rank) start = s;
      s = make_float2(fmaf(q.x, s.x, q.y), fmaf(q.z, s.y, q.w));
    }
  }
  carry = s;
  return make_float2(fmaf(before.x, start.x, before.y), fmaf(before.z, start.y, before.w));
}

// Appends the map (a, b) of one row to m, for both channels.
__device__ __forceinline__ void rec_append(float4& m, float2 a, float2 b) {
  m = make_float4(m.x * a.x, fmaf(a.x, m.y, b.x), m.z * a.y, fmaf(a.y, m.w, b.y));
}

template <class T, bool GATE, class G>
__global__ void __launch_bounds__(G::NT, 2) rec_forward_kernel(const __grid_constant__ RecArgs<T> a, unsigned C) {
  constexpr int R = G::R, NA = GATE ? 3 : 2;
  extern __shared__ __align__(16) unsigned char tiles[];
  __shared__ RecShared sh;
  pdl_entry();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned rank = C > 1 ? cluster_rank() : 0;
  const unsigned strip = blockIdx.x / C;
  const long long b = strip / a.strips;
  const int d0 = (int)(strip % a.strips) * G::W, ch = d0 + 2 * lane;
  const long long step = (long long)C * G::L, rounds = (a.T_ + step - 1) / step;
  const long long tile0 = (long long)rank * G::L;
  const RecStrip<T> x = {a.x + b * a.xb + d0, a.xt}, f = {a.f + b * a.fb + d0, a.ft},
                    g = {GATE ? a.i + b * a.ib + d0 : nullptr, a.it};
  T* y = a.y + b * a.yb + ch;
  const uint8_t* starts = a.starts ? a.starts + b * a.T_ : nullptr;

  auto fetch = [&](long long k) {  // this CTA's tile of round k; one commit group a round
    if (k < rounds) {
      unsigned char* base = tiles + (size_t)(k % G::STAGES) * NA * G::ARRAY;
#pragma unroll
      for (int n = 0; n < G::ITERS; ++n) {
        const int at = tid + n * G::NT, r = at / G::CHUNKS, c = at % G::CHUNKS;
        if (G::EDGE && r >= G::L) break;
        const long long t = tile0 + k * step + r;
        const bool on = t < a.T_;
        rec_copy<T, G>(base, x, r, c, t, on, d0, a.D);
        rec_copy<T, G>(base + G::ARRAY, f, r, c, t, on, d0, a.D);
        if constexpr (GATE) rec_copy<T, G>(base + 2 * G::ARRAY, g, r, c, t, on, d0, a.D);
      }
    }
    cp_async_commit();
  };
  auto flags = [&](long long k) -> int {  // lane r < R: whether its warp's row r is a start
    const long long t = tile0 + k * step + warp * R + lane;
    return starts && lane < R && t < a.T_ ? starts[t] : 0;
  };
#pragma unroll
  for (int k = 0; k < G::STAGES - 1; ++k) fetch(k);
  int flag = flags(0);
  float2 carry = make_float2(0.f, 0.f);
  if (a.h0) {
    if (ch < a.D) carry.x = a.h0[b * a.D + ch];
    if (ch + 1 < a.D) carry.y = a.h0[b * a.D + ch + 1];
  }
  if (C > 1) cluster_sync();  // the others are there to be written to

  for (long long k = 0; k < rounds; ++k) {
    const long long t0 = tile0 + k * step + warp * R;
    cp_async_wait<G::STAGES - 2>();
    __syncthreads();  // the tile is in; the one before it has been read by all
    fetch(k + G::STAGES - 1);
    const unsigned drop = __ballot_sync(0xffffffffu, flag != 0);
    flag = flags(k + 1);
    const unsigned char* base = tiles + (size_t)(k % G::STAGES) * NA * G::ARRAY;
    float2 av[R], bv[R];
    float4 m = make_float4(1.f, 0.f, 1.f, 0.f);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      // Past the end the map is the identity, so that `carry` ends as the last state.
      av[r] = make_float2(1.f, 1.f);
      bv[r] = make_float2(0.f, 0.f);
      if (t0 + r < a.T_) {
        const int row = warp * R + r;
        const float2 xs = rec_pair<T, G>(base, x, row, lane, t0 + r);
        const float2 fs = rec_pair<T, G>(base + G::ARRAY, f, row, lane, t0 + r);
        float2 u;
        if constexpr (GATE) {
          const float2 is = rec_pair<T, G>(base + 2 * G::ARRAY, g, row, lane, t0 + r);
          av[r] = make_float2(sigmoid(fs.x), sigmoid(fs.y));
          u = make_float2(sigmoid(is.x), sigmoid(is.y));
        } else {
          sigmoid_both(fs.x, av[r].x, u.x);
          sigmoid_both(fs.y, av[r].y, u.y);
        }
        if (drop >> r & 1) av[r] = make_float2(0.f, 0.f);
        bv[r] = make_float2(u.x * xs.x, u.y * xs.y);
      }
      rec_append(m, av[r], bv[r]);
    }
    float2 s = rec_exchange(m, carry, sh, C, rank, (int)(k & 1));
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (t0 + r < a.T_) {
        s = make_float2(fmaf(av[r].x, s.x, bv[r].x), fmaf(av[r].y, s.y, bv[r].y));
        rec_store<T, G::EDGE>(y + (t0 + r) * a.yt, s, ch, a.D);
      }
    }
  }
  if (a.last && rank == 0 && warp == 0) {
    if (ch < a.D) a.last[b * a.D + ch] = carry.x;
    if (ch + 1 < a.D) a.last[b * a.D + ch + 1] = carry.y;
  }
}

// Position p = 0, 1, ... counts rows from the end: t = T - 1 - p.
template <class T, bool GATE, class G>
__global__ void __launch_bounds__(G::NT, 2) rec_backward_kernel(const __grid_constant__ RecArgs<T> a, unsigned C) {
  constexpr int R = G::R, NA = GATE ? 5 : 4;
  extern __shared__ __align__(16) unsigned char tiles[];
  __shared__ RecShared sh;
  pdl_entry();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned rank = C > 1 ? cluster_rank() : 0;
  const unsigned strip = blockIdx.x / C;
  const long long b = strip / a.strips;
  const int d0 = (int)(strip % a.strips) * G::W, ch = d0 + 2 * lane;
  const long long step = (long long)C * G::L, rounds = (a.T_ + step - 1) / step;
  const long long tile0 = (long long)rank * G::L;
  const RecStrip<T> f = {a.f + b * a.fb + d0, a.ft}, dh = {a.dh + b * a.dhb + d0, a.dht},
                    x = {a.x + b * a.xb + d0, a.xt}, h = {a.h + b * a.hb + d0, a.ht},
                    g = {GATE ? a.i + b * a.ib + d0 : nullptr, a.it};
  T *dx = a.dx + b * a.dxb + ch, *df = a.df + b * a.dfb + ch, *di = GATE ? a.di + b * a.dib + ch : nullptr;
  const uint8_t* starts = a.starts ? a.starts + b * a.T_ : nullptr;

  auto fetch = [&](long long k) {
    if (k < rounds) {
      unsigned char* base = tiles + (size_t)(k % G::STAGES) * NA * G::ARRAY;
#pragma unroll
      for (int n = 0; n < G::ITERS; ++n) {
        const int at = tid + n * G::NT, r = at / G::CHUNKS, c = at % G::CHUNKS;
        if (G::EDGE && r >= G::L) break;
        const long long t = a.T_ - 1 - (tile0 + k * step + r);
        const bool on = t >= 0;
        rec_copy<T, G>(base, f, r, c, t, on, d0, a.D);
        rec_copy<T, G>(base + G::ARRAY, dh, r, c, t, on, d0, a.D);
        rec_copy<T, G>(base + 2 * G::ARRAY, x, r, c, t, on, d0, a.D);
        rec_copy<T, G>(base + 3 * G::ARRAY, h, r, c, t - 1, t > 0, d0, a.D);
        if constexpr (GATE) rec_copy<T, G>(base + 4 * G::ARRAY, g, r, c, t, on, d0, a.D);
      }
    }
    cp_async_commit();
  };
  auto flags = [&](long long k) -> int {
    const long long t = a.T_ - 1 - (tile0 + k * step + warp * R + lane);
    return starts && lane < R && t >= 0 ? starts[t] : 0;
  };
#pragma unroll
  for (int k = 0; k < G::STAGES - 1; ++k) fetch(k);
  int flag = flags(0);
  float2 carry = make_float2(0.f, 0.f), first = carry;
  if (a.dlast) {
    if (ch < a.D) carry.x = a.dlast[b * a.D + ch];
    if (ch + 1 < a.D) carry.y = a.dlast[b * a.D + ch + 1];
  }
  if (a.h0) {
    if (ch < a.D) first.x = a.h0[b * a.D + ch];
    if (ch + 1 < a.D) first.y = a.h0[b * a.D + ch + 1];
  }
  if (C > 1) cluster_sync();

  for (long long k = 0; k < rounds; ++k) {
    const long long t0 = a.T_ - 1 - (tile0 + k * step + warp * R);  // this warp's rows: t0, t0 - 1, ...
    cp_async_wait<G::STAGES - 2>();
    __syncthreads();
    fetch(k + G::STAGES - 1);
    const unsigned drop = __ballot_sync(0xffffffffu, flag != 0);
    flag = flags(k + 1);
    const unsigned char* base = tiles + (size_t)(k % G::STAGES) * NA * G::ARRAY;
    float2 s[R], s1[R];  // sigmoid(f) and 1 - sigmoid(f)
    float4 m = make_float4(1.f, 0.f, 1.f, 0.f);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[r] = s1[r] = make_float2(0.f, 0.f);
      if (t0 - r >= 0) {
        const int row = warp * R + r;
        const float2 fs = rec_pair<T, G>(base, f, row, lane, t0 - r);
        const float2 ds = rec_pair<T, G>(base + G::ARRAY, dh, row, lane, t0 - r);
        sigmoid_both(fs.x, s[r].x, s1[r].x);
        sigmoid_both(fs.y, s[r].y, s1[r].y);
        const float2 av = drop >> r & 1 ? make_float2(0.f, 0.f) : s[r];
        rec_append(m, av, make_float2(av.x * ds.x, av.y * ds.y));
      }
    }
    float2 c = rec_exchange(m, carry, sh, C, rank, (int)(k & 1));  // c_{t+1} of the warp's first row
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long t = t0 - r;
      if (t < 0) break;
      const int row = warp * R + r;
      const float2 ds = rec_pair<T, G>(base + G::ARRAY, dh, row, lane, t);
      const float2 xs = rec_pair<T, G>(base + 2 * G::ARRAY, x, row, lane, t);
      float2 hs = t > 0 ? rec_pair<T, G>(base + 3 * G::ARRAY, h, row, lane, t - 1) : first;
      const bool dropped = drop >> r & 1;
      if (dropped) hs = make_float2(0.f, 0.f);
      const float2 gt = make_float2(ds.x + c.x, ds.y + c.y);  // dL/dh_t
      const float2 fg = make_float2(s[r].x * s1[r].x * gt.x, s[r].y * s1[r].y * gt.y);
      if constexpr (GATE) {
        const float2 is = rec_pair<T, G>(base + 4 * G::ARRAY, g, row, lane, t);
        float2 u, u1;
        sigmoid_both(is.x, u.x, u1.x);
        sigmoid_both(is.y, u.y, u1.y);
        const float2 ug = make_float2(u.x * gt.x, u.y * gt.y);
        rec_store<T, G::EDGE>(dx + t * a.dxt, ug, ch, a.D);
        rec_store<T, G::EDGE>(df + t * a.dft, make_float2(fg.x * hs.x, fg.y * hs.y), ch, a.D);
        rec_store<T, G::EDGE>(di + t * a.dit, make_float2(ug.x * u1.x * xs.x, ug.y * u1.y * xs.y), ch, a.D);
      } else {
        rec_store<T, G::EDGE>(dx + t * a.dxt, make_float2(s1[r].x * gt.x, s1[r].y * gt.y), ch, a.D);
        rec_store<T, G::EDGE>(df + t * a.dft, make_float2(fg.x * (hs.x - xs.x), fg.y * (hs.y - xs.y)), ch, a.D);
      }
      c = dropped ? make_float2(0.f, 0.f) : make_float2(s[r].x * gt.x, s[r].y * gt.y);
    }
  }
  if (a.dh0 && rank == 0 && warp == 0) {
    if (ch < a.D) a.dh0[b * a.D + ch] = carry.x;
    if (ch + 1 < a.D) a.dh0[b * a.D + ch + 1] = carry.y;
  }
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

template <class G, int NA, class T, class K>
cudaError_t rec_launch(K kernel, const RecurrenceJob& j, RecArgs<T> a, const LaunchCtx& ctx) {
  const long long strips = (j.D + G::W - 1) / G::W;
  const unsigned C = rec_cluster<G>(strips * j.B, j.T, ctx.num_sms);
  a.strips = (int)strips;
  constexpr int smem = G::STAGES * NA * G::ARRAY;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  profile_before(ctx);
  e = launch_pdl_cluster(kernel, (unsigned)(strips * j.B * C), G::NT, C, smem, ctx.stream, a, C);
  profile_after(ctx);
  return e;
}

template <class T, bool EDGE> cudaError_t rec_forward(const RecurrenceJob& j, const LaunchCtx& ctx) {
  using G = RecGeom<T, EDGE, 3>;
  const RecArgs<T> a = rec_args<T>(j);
  return j.i.p ? rec_launch<G, 3>(rec_forward_kernel<T, true, G>, j, a, ctx)
               : rec_launch<G, 2>(rec_forward_kernel<T, false, G>, j, a, ctx);
}
template <class T, bool EDGE> cudaError_t rec_backward(const RecurrenceJob& j, const LaunchCtx& ctx) {
  using G = RecGeom<T, EDGE, 2>;
  const RecArgs<T> a = rec_args<T>(j);
  return j.i.p ? rec_launch<G, 5>(rec_backward_kernel<T, true, G>, j, a, ctx)
               : rec_launch<G, 4>(rec_backward_kernel<T, false, G>, j, a, ctx);
}

template <class T> cudaError_t launch_recurrence(const RecurrenceJob& j, const LaunchCtx& ctx) {
  bool even = j.D % (16 / sizeof(T)) == 0;
  for (const SeqArray* s : {&j.x, &j.f, &j.i, &j.h}) even = even && rows16<T>(*s, j.B, j.T);
  return even ? rec_forward<T, false>(j, ctx) : rec_forward<T, true>(j, ctx);
}

template <class T> cudaError_t launch_recurrence_backward(const RecurrenceJob& j, const LaunchCtx& ctx) {
  bool even = j.D % (16 / sizeof(T)) == 0;
  for (const SeqArray* s : {&j.x, &j.f, &j.i, &j.h, &j.dh, &j.dx, &j.df, &j.di}) even = even && rows16<T>(*s, j.B, j.T);
  return even ? rec_backward<T, false>(j, ctx) : rec_backward<T, true>(j, ctx);
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
