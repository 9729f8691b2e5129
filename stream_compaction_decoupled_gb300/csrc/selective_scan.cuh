// selective_scan.cuh -- the selective state space scan, its gradient, and its form for one token
// a call on a pool of states.
//
//   D_t = softplus(dt_t + bias),  a_t = exp(D_t A),  h_t = a_t h_{t-1} + D_t x_t B_t,
//   y_t = (C_t . h_t + d x_t) silu(z_t)
//
// for each channel, with N states h a channel; B and C (N values a token) are shared by the
// channels of a group.  A document start drops h_{t-1} (by selection: also infinities and NaNs).
// The gradient, with e_t = dy_t silu(z_t) and carry_t what token t + 1 passes back:
//   g_t = C_t e_t + carry_t,   q_t = a_t g_t h_{t-1},   carry_{t-1} = a_t g_t (0 at a start),
//   dC_t = sum over channels of e_t h_t,      dB_t = sum over channels of g_t D_t x_t,
//   dx_t = d e_t + D_t (B_t . g_t),           dD_t = x_t (B_t . g_t) + q_t . A,
//   dA = sum_t q_t D_t,  dz_t = dy_t (C_t . h_t + d x_t) silu'(z_t),  ddt_t = dD_t sigmoid(dt_t + bias).
//
// Bound by issue: an exponential and four fp32 operations for each state and token, against 8
// bytes a token and channel (16 bits).  Forward, a warp is on its own: 64 / LN channels of one
// group, LN lanes a pair of channels and 16 / LN states of both a lane (more than 16 states in
// blocks of 16), so that a token's B and C, the same for all channels, are read once for 32 / LN
// states and tokens a lane.  (A 128-bit read of shared memory costs four passes even where all
// lanes read the same; reading B and C for 4 states of 2 channels with each value twice took 24
// passes a token and a quarter of the time.)  What is done once a token and channel (softplus,
// gate, conversions) goes around the lanes of a pair, a token each.  Inputs come through a ring of
// asynchronous copies, their start flags 32 tiles at a time.
//
// The gradient: a block of 128 threads takes 64 channels and tiles of 16 tokens, in three phases:
//   A  a lane takes two neighbouring channels, a warp 4 tokens: D, D x to shared memory;
//   B  a warp takes 16 channels and all 16 tokens: a thread 2 channels and 4 states of each block
//      of 16, 4 lanes a channel; its part of the sums over states to shared memory;
//   C  as A: the four lanes' parts are summed, then what is done once a token and channel.
//
// The tokens of a row are one chain.  Where the rows and channels are too few for the device,
// they are split into parts: a first kernel finds what each part makes of a state of zero, and
// with exp(A sum D) each part knows where it starts (the gradient: from the other end).
//
// Measured (GB300): 8 x 2048 x 2048, 16 states, bf16, gated, with starts and kept states 285 us;
// 1 x 32768 x 2048 continued 511 us.
#pragma once

#include "lm.cuh"
#include "lm.h"

namespace gbs {

constexpr int kSscThreads = 128;
constexpr int kSscRows = kSscTile / 4;  // tokens of a warp in phases A and C

template <class T> struct SscArgs {
  const T *x, *dt, *z, *b, *c, *dy;
  T *y, *dx, *ddt, *dz;
  long long xb, xt, dtb, dtt, zb, zt, yb, yt, dyb, dyt, dxb, dxt, ddtb, ddtt, dzb, dzt;
  long long bb, bt, bg, cb, ct, cg;
  const float *a, *d, *bias, *h0, *dlast;
  const uint8_t* starts;
  float *last, *kept, *dh0;
  // Scratch: what a part makes of a state of zero (B, parts - 1, D, N), its sum of D (B, parts
  // - 1, D), whether it drops what came before it (B, parts - 1).
  float *ends, *sums, *drops;
  // Gradient: parts of dB, dC (blocks, B, T, G, N) and of dA, dd, dbias (B parts, D, N + 2).
  float *part_b, *part_c, *part_a;
  long long B;
  int T_, D, N, NP, G, DG, blocks, parts, part_tiles, tiles, softplus;
  bool vec;     // (D, N) arrays can be read and written in 16-byte pieces
};

// Two neighbouring channels of a row, as they lie in memory.
template <class T, bool EDGE> struct SscPair {
  using Raw = std::conditional_t<sizeof(T) == 2, unsigned, float2>;
  static __device__ __forceinline__ Raw load(const T* p, int count) {
    Raw r;
    if constexpr (sizeof(T) == 4) r = make_float2(0.f, 0.f);
    else r = 0u;
    if constexpr (EDGE) {
      T v[2] = {narrow<T>(0.f), narrow<T>(0.f)};
      if (count > 0) v[0] = p[0];
      if (count > 1) v[1] = p[1];
      memcpy(&r, v, sizeof(r));
    } else {
      if (count > 0) r = *(const Raw*)p;
    }
    return r;
  }
  static __device__ __forceinline__ void store(T* p, int count, float2 f) {
    Raw r;
    if constexpr (sizeof(T) == 4) r = f;
    else r = narrow2<T>(f);
    if constexpr (EDGE) {
      T v[2];
      memcpy(v, &r, sizeof(r));
      if (count > 0) p[0] = v[0];
      if (count > 1) p[1] = v[1];
    } else {
      if (count > 0) *(Raw*)p = r;
    }
  }
  static __device__ __forceinline__ float2 wide(Raw r) {
    if constexpr (sizeof(T) == 4) return r;
    else return widen2<T>(r);
  }
};

// Where a block works, and which channels and states a thread has.
template <class T> struct SscPlace {
  long long b;         // batch row
  int group, block;    // of channels, and the block of 64 within it
  int part;            // of the tokens
  int tile0, tile1;    // its tiles
  int lane, warp;
  int ch;              // phases A and C: the lane's first channel, and how many of its two exist
  int count;
  int pr, ln;          // phase B: the thread's pair of channels within the block, its place among 4 lanes
  int chb, countb;
  __device__ __forceinline__ SscPlace(const SscArgs<T>& a, int first_part, int parts) {
    long long u = blockIdx.x;
    block = (int)(u % a.blocks);
    u /= a.blocks;
    group = (int)(u % a.G);
    u /= a.G;
    part = first_part + (int)(u % parts);
    b = u / parts;
    tile0 = part * a.part_tiles;
    tile1 = min(a.tiles, tile0 + a.part_tiles);
    lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int left = min(kSscChannels, a.DG - block * kSscChannels), base = group * a.DG + block * kSscChannels;
    ch = base + 2 * lane;
    count = min(2, left - 2 * lane);
    pr = warp * 8 + (lane >> 2);
    ln = lane & 3;
    chb = base + 2 * pr;
    countb = min(2, left - 2 * pr);
  }
};

// State s (0 .. 3) of a thread in the block of 16 from n0: the lanes' pairs lie side by side.
__device__ __forceinline__ int ssc_state(int n0, int ln, int s) { return n0 + (s >> 1) * 8 + ln * 2 + (s & 1); }

// Values (channel, state) of a (D, N) array for the thread's pair of channels; `other` where
// there are none.
__device__ __forceinline__ float2 ssc_load(const float* p, int n, int N, int count, float other) {
  float2 v = make_float2(other, other);
  if (n < N) {
    if (count > 0) v.x = p[n];
    if (count > 1) v.y = p[N + n];
  }
  return v;
}
__device__ __forceinline__ void ssc_store(float* p, int n, int N, int count, float2 v) {
  if (n < N) {
    if (count > 0) p[n] = v.x;
    if (count > 1) p[N + n] = v.y;
  }
}
// exp of the product, a in units of log2 e.  In single operations: a packed product before the
// exponential costs more than the instruction it saves (measured in a loop of nothing else, 32
// states a thread, 3 warps a scheduler: 6.9 cycles a state and token with packed products and sums,
// 5.2 with these and the sums single and only D x B packed, 5.9 with all of it single).
__device__ __forceinline__ float2 ssc_decay(float2 a, float2 d) { return make_float2(ex2(a.x * d.x), ex2(a.y * d.y)); }
__device__ __forceinline__ float2 ssc_fma(float2 a, float2 b, float2 c) { return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)); }
// The thread's A in units of log2 e.
template <class T>
__device__ __forceinline__ void ssc_rates(const SscArgs<T>& a, const SscPlace<T>& at, int n0, float2 (&r)[4]) {
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const float2 v = ssc_load(a.a + (long long)at.chb * a.N, ssc_state(n0, at.ln, s), a.N, at.countb, 0.f);
    r[s] = mul2(v, make_float2(kLog2e, kLog2e));
  }
}
// Bit t: token t of the tile starts a document.
template <class T> __device__ __forceinline__ unsigned ssc_starts(const SscArgs<T>& a, long long b, int t0, int lane) {
  if (!a.starts) return 0;
  const bool s = lane < kSscTile && t0 + lane < a.T_ && a.starts[b * a.T_ + t0 + lane] != 0;
  return __ballot_sync(0xffffffffu, s);
}
// A tile's values of B or C, each twice, to shared memory (tokens, NP), zero where there are none.
template <class T>
__device__ __forceinline__ void ssc_vectors(const SscArgs<T>& a, const T* p, long long stride, int t0, int NP, float2* out) {
  const int total = kSscTile * NP;
  for (int k = threadIdx.x; k < total; k += kSscThreads) {
    const int t = k / NP, n = k % NP;
    const float v = n < a.N && t0 + t < a.T_ ? widen(p[t * stride + n]) : 0.f;
    out[k] = make_float2(v, v);
  }
}
template <class T> __device__ __forceinline__ float2 ssc_step_size(const SscArgs<T>& a, float2 v) {
  return a.softplus ? softplus2<T>(v) : v;
}
// The two 16-byte halves of a pair's four parts, placed so that neither the writes (4 lanes
// of 8 bytes a pair) nor the reads (a lane a pair) meet in a bank.
__device__ __forceinline__ int ssc_half(int pair, int half) { return half ^ ((pair >> 2) & 1); }
__device__ __forceinline__ void ssc_put(float2* part, int t, int pair, int ln, float2 v) {
  part[(t * 32 + pair) * 4 + ssc_half(pair, ln >> 1) * 2 + (ln & 1)] = v;
}
__device__ __forceinline__ float2 ssc_get(const float2* part, int t, int pair) {
  const float4* p = (const float4*)(part + (t * 32 + pair) * 4);
  const float4 lo = p[ssc_half(pair, 0)], hi = p[ssc_half(pair, 1)];
  return add2(add2(make_float2(lo.x, lo.y), make_float2(lo.z, lo.w)), add2(make_float2(hi.x, hi.y), make_float2(hi.z, hi.w)));
}

// The state before a part: what comes in, through each part before it in turn (`first` to
// `last`, either way).
template <class T>
__device__ __forceinline__ float2 ssc_through(const SscArgs<T>& a, const SscPlace<T>& at, int n, float2 rate, float2 h,
                                              int first, int count, int step) {
  int p = first;
#pragma unroll 4
  for (int k = 0; k < count; ++k, p += step) {
    const long long row = at.b * (a.parts - 1) + p;
    const float2 e = ssc_load(a.ends + (row * a.D + at.chb) * a.N, n, a.N, at.countb, 0.f);
    const float* s = a.sums + row * a.D + at.chb;
    const float2 sum = make_float2(at.countb > 0 ? s[0] : 0.f, at.countb > 1 ? s[1] : 0.f);
    h = a.drops[row] != 0.f ? e : fma2(ssc_decay(rate, sum), h, e);
  }
  return h;
}

// The part's sum of D: each thread's own over its tokens, summed over the warps.
template <class T>
__device__ __forceinline__ void ssc_write_sums(const SscArgs<T>& a, const SscPlace<T>& at, float2 sum, bool dropped, long long row,
                                               float2* scratch) {
  scratch[at.warp * 32 + at.lane] = sum;
  __syncthreads();
  if (at.warp == 0) {
    const float2 s = add2(add2(scratch[at.lane], scratch[32 + at.lane]), add2(scratch[64 + at.lane], scratch[96 + at.lane]));
    float* p = a.sums + row * a.D + at.ch;
    if (at.count > 0) p[0] = s.x;
    if (at.count > 1) p[1] = s.y;
    if (at.lane == 0 && at.block == 0 && at.group == 0) a.drops[row] = dropped ? 1.f : 0.f;
  }
}

// Shared memory, in float2: D and D x of the tile (2), [e (1)], the parts of sums over states (4
// for each of SUMS), B and C, and with more than 16 states what a thread keeps of each block.
struct SscShared {
  static constexpr int kDx = kSscTile * 32 * 2, kE = kSscTile * 32, kPart = kSscTile * 32 * 4;
  static constexpr int kSave = 3 * 4 * kSscThreads, kRed = kSscTile * 4 * 32 / 2;
  static size_t forward(int NP, bool ends) {
    return 8 * ((size_t)kDx + (ends ? 0 : kPart) + kSscTile * NP * (ends ? 1 : 2) + (NP > 16 ? NP / 16 * 4 * kSscThreads : 0)) +
           (ends ? 8 * 128 : 0);
  }
  static size_t carry(int NP) {
    return 8 * ((size_t)kDx + kE + kSscTile * NP + (NP > 16 ? NP / 16 * 4 * kSscThreads : 0) + 128);
  }
  static size_t backward(int NP) {
    return 8 * ((size_t)kDx + kE + 3 * kPart + kSave + kRed + kSscTile * NP * 2 + (NP > 16 ? 2 * (NP / 16) * 4 * kSscThreads : 0));
  }
};

// ---- forward ---------------------------------------------------------------------------

// M = 16 / LN states of two channels a thread, LN lanes a pair of channels; a warp is on its own:
// WIDTH channels, tiles of L tokens, of which a lane prepares and finishes R.  What a warp reads
// comes by asynchronous copies into a ring of STAGES tiles of its own in shared memory.
template <class T, bool EDGE_, int LN_> struct SscLane {
  static constexpr bool EDGE = EDGE_;
  static constexpr int LN = LN_, L = 8, R = L / LN, M = 16 / LN, WIDTH = 64 / LN;
  static constexpr int STAGES = sizeof(T) == 2 ? 3 : 2;
  static constexpr int ROW = WIDTH * (int)sizeof(T), ARRAY = L * ROW;  // bytes
  static constexpr int VECTORS = L * 32 * (int)sizeof(T);               // B and C of 16 states, as they are
  static constexpr int CHUNKS = ROW / 16;                               // 16-byte copies of a row
  using P = SscPair<T, EDGE>;
  using Raw = typename P::Raw;
  static __host__ __device__ constexpr int stage_bytes(int NB) { return 3 * ARRAY + NB * VECTORS; }
  // Bytes a warp: the ring, B and C widened, D and D x of each pair, and with more than 16 states
  // those of each block.
  static __host__ __device__ constexpr int warp_bytes(int NB) {
    return STAGES * stage_bytes(NB) + NB * L * 32 * 4 + L * (32 / LN) * 16 + (NB > 1 ? NB * 2 * M * 32 * 4 : 0);
  }
};

// Where a warp works.
template <class T> struct SscWarp {
  long long b;
  int group, part, t0, t1;  // tokens of its part
  int base, width;          // the warp's first channel, and how many it has
  int ch, count;            // the lane's first channel, and how many of its two exist
  bool idle;
  __device__ __forceinline__ SscWarp(const SscArgs<T>& a, int LN, int parts) {
    const int lane = threadIdx.x & 31, most = 64 / LN, blocks = (a.DG + most - 1) / most;
    long long u = (long long)blockIdx.x * (kSscThreads / 32) + (threadIdx.x >> 5);
    const int block = (int)(u % blocks);
    u /= blocks;
    group = (int)(u % a.G);
    u /= a.G;
    part = (int)(u % parts);
    b = u / parts;
    idle = b >= a.B;
    t0 = part * a.part_tiles * kSscTile;
    t1 = (int)min((long long)a.T_, (long long)t0 + (long long)a.part_tiles * kSscTile);
    base = group * a.DG + block * most;
    width = min(most, (group + 1) * a.DG - base);
    ch = base + 2 * (lane / LN);
    count = min(2, base + width - ch);
    if (count <= 0) ch = base;  // what it loads is real, what it makes is not stored
  }
};

// M values of two channels of a (D, N) array, in pairs of states; `other` where there are none.
template <int M, bool VEC> __device__ __forceinline__ void ssc_load_states(const float* p, int n0, int N, int count, float2 (&v)[2][M / 2]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
#pragma unroll
    for (int j = 0; j < M / 4; ++j) {
      float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
      const int n = n0 + 4 * j;
      const float* at = p + (long long)c * N + n;
      if (VEC) {
        if (c < count && n < N) q = *(const float4*)at;
      } else if (c < count) {
        if (n < N) q.x = at[0];
        if (n + 1 < N) q.y = at[1];
        if (n + 2 < N) q.z = at[2];
        if (n + 3 < N) q.w = at[3];
      }
      v[c][2 * j] = make_float2(q.x, q.y);
      v[c][2 * j + 1] = make_float2(q.z, q.w);
    }
  }
}
template <int M, bool VEC> __device__ __forceinline__ void ssc_store_states(float* p, int n0, int N, int count, const float2 (&v)[2][M / 2]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
#pragma unroll
    for (int j = 0; j < M / 4; ++j) {
      const int n = n0 + 4 * j;
      const float4 q = make_float4(v[c][2 * j].x, v[c][2 * j].y, v[c][2 * j + 1].x, v[c][2 * j + 1].y);
      float* at = p + (long long)c * N + n;
      if (VEC) {
        if (c < count && n < N) *(float4*)at = q;
      } else if (c < count) {
        if (n < N) at[0] = q.x;
        if (n + 1 < N) at[1] = q.y;
        if (n + 2 < N) at[2] = q.z;
        if (n + 3 < N) at[3] = q.w;
      }
    }
  }
}
template <int M> __device__ __forceinline__ void ssc_load_any(bool vec, const float* p, int n0, int N, int count, float2 (&v)[2][M / 2]) {
  if (vec) ssc_load_states<M, true>(p, n0, N, count, v);
  else ssc_load_states<M, false>(p, n0, N, count, v);
}
template <int M> __device__ __forceinline__ void ssc_store_any(bool vec, float* p, int n0, int N, int count, const float2 (&v)[2][M / 2]) {
  if (vec) ssc_store_states<M, true>(p, n0, N, count, v);
  else ssc_store_states<M, false>(p, n0, N, count, v);
}

// ENDS: only the states that the part ends with, from a state of zero, and its sum of D.
template <class T, bool EDGE, bool ONE, bool ENDS, int LN>
__global__ void __launch_bounds__(kSscThreads, 4) ssc_forward_kernel(const __grid_constant__ SscArgs<T> a) {
  pdl_entry();
  using S = SscLane<T, EDGE, LN>;
  using P = typename S::P;
  constexpr int L = S::L, R = S::R, M = S::M;
  extern __shared__ __align__(16) float2 ssc_shared[];
  const int NB = ONE ? 1 : a.NP / 16;
  const int lane = threadIdx.x & 31, ln = lane % LN;
  unsigned char* ring = (unsigned char*)ssc_shared + (threadIdx.x >> 5) * S::warp_bytes(NB);
  const int stage_bytes = S::stage_bytes(NB);
  float* vs = (float*)(ring + S::STAGES * stage_bytes);  // B (16) and C (16) of each block's tokens
  float4* ds = (float4*)(vs + NB * L * 32);           // D and D x (token, pair)
  float4* hs = ds + L * (32 / LN);                    // states by block, where there are several
  const SscWarp<T> at(a, LN, ENDS ? a.parts - 1 : a.parts);
  if (at.idle) return;
  const float2 zero = make_float2(0.f, 0.f);
  const long long row = at.b * a.D + at.ch;  // of (B, D, N) arrays

  float2 rate[2][M / 2], h[2][M / 2];
  const auto rates = [&](int k) {
    ssc_load_any<M>(a.vec, a.a + (long long)at.ch * a.N, k * 16 + ln * M, a.N, at.count, rate);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int j = 0; j < M / 2; ++j) rate[c][j] = mul2(rate[c][j], make_float2(kLog2e, kLog2e));
  };
  const auto put_h = [&](int k) {
#pragma unroll
    for (int j = 0; j < M / 2; ++j) hs[(k * M / 2 + j) * 32 + lane] = make_float4(h[0][j].x, h[0][j].y, h[1][j].x, h[1][j].y);
  };
  const auto get_h = [&](int k) {
#pragma unroll
    for (int j = 0; j < M / 2; ++j) {
      const float4 q = hs[(k * M / 2 + j) * 32 + lane];
      h[0][j] = make_float2(q.x, q.y), h[1][j] = make_float2(q.z, q.w);
    }
  };
  for (int k = 0; k < NB; ++k) {
    rates(k);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int j = 0; j < M / 2; ++j) h[c][j] = zero;
    if constexpr (!ENDS) {
      if (a.h0) ssc_load_any<M>(a.vec, a.h0 + row * a.N, k * 16 + ln * M, a.N, at.count, h);
      // Through the parts before this one in turn.
      for (int p = 0; p < at.part; ++p) {
        const long long pr = at.b * (a.parts - 1) + p;
        float2 e[2][M / 2];
        ssc_load_any<M>(a.vec, a.ends + (pr * a.D + at.ch) * a.N, k * 16 + ln * M, a.N, at.count, e);
        const float* s = a.sums + pr * a.D + at.ch;
        const float sum[2] = {at.count > 0 ? s[0] : 0.f, at.count > 1 ? s[1] : 0.f};
        const bool dropped = a.drops[pr] != 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < M / 2; ++j)
            h[c][j] = dropped ? e[c][j] : fma2(ssc_decay(rate[c][j], make_float2(sum[c], sum[c])), h[c][j], e[c][j]);
      }
    }
    if constexpr (!ONE) put_h(k);
  }
  float2 bias = zero, skip = zero, sum = zero;
  if (a.bias) bias = make_float2(at.count > 0 ? a.bias[at.ch] : 0.f, at.count > 1 ? a.bias[at.ch + 1] : 0.f);
  if (!ENDS && a.d) skip = make_float2(at.count > 0 ? a.d[at.ch] : 0.f, at.count > 1 ? a.d[at.ch + 1] : 0.f);

  // The lane's own tokens of a tile are those with (t % LN) = ln.
  const T* px = a.x + at.b * a.xb;
  const T* pdt = a.dt + at.b * a.dtb;
  const bool gated = !ENDS && a.z;
  const T* pz = gated ? a.z + at.b * a.zb : nullptr;
  T* py = ENDS ? nullptr : a.y + at.b * a.yb + (long long)(at.t0 + ln) * a.yt + at.ch;
  const int n = lane & 15;
  const bool second = !ENDS && lane >= 16;
  const T* pb = a.b + at.b * a.bb + at.group * a.bg;
  const T* pc = ENDS ? pb : a.c + at.b * a.cb + at.group * a.cg;
  const T* pv = second ? pc : pb;
  const long long sv = second ? a.ct : a.bt;
  const uint8_t* ps = a.starts ? a.starts + at.b * a.T_ : nullptr;

  // Starts a tile's copies into the ring.  EDGE, where they cannot be in pieces of 16 bytes: loads
  // the tile, for `put` to store behind the one that is worked on.  (No ordinary load goes among
  // the copies: waiting for it would be waiting for them.)
  constexpr int V = 16 / sizeof(T), PER = 32 / V;
  const int own_row = lane / S::CHUNKS, own_c = lane % S::CHUNKS * V;   // the lane's pieces of x, dt, z
  const int v_row = lane / PER, v_c = lane % PER * V;                   // and of B or C
  const bool copies = lane < L * S::CHUNKS && own_c < at.width;
  const T* qx = px + (long long)(at.t0 + own_row) * a.xt + at.base + own_c;
  const T* qd = pdt + (long long)(at.t0 + own_row) * a.dtt + at.base + own_c;
  const T* qz = gated ? pz + (long long)(at.t0 + own_row) * a.zt + at.base + own_c : nullptr;
  const long long qs = v_c < 16 ? a.bt : a.ct;
  const T* qv = (v_c < 16 ? pb : pc) + (long long)(at.t0 + v_row) * qs + v_c % 16;
  typename S::Raw ex[EDGE ? R : 1], ed[EDGE ? R : 1], ez[EDGE ? R : 1];
  T ev[EDGE && ONE ? L : 1];
  const auto get = [&](int t, int stage) {
    unsigned char* to_stage = ring + stage * stage_bytes;
    if (t < at.t1) {
      if constexpr (EDGE) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const long long row = min(t + ln + r * LN, a.T_ - 1);
          ex[r] = P::load(px + row * a.xt + at.ch, at.count);
          ed[r] = P::load(pdt + row * a.dtt + at.ch, at.count);
          if (gated) ez[r] = P::load(pz + row * a.zt + at.ch, at.count);
        }
        if constexpr (ONE) {
#pragma unroll
          for (int i = 0; i < L; ++i) ev[i] = pv[(long long)min(t + i, a.T_ - 1) * sv + (n < a.N ? n : 0)];
        }
      } else {
        // Rows behind the last are read as the last: that many rows back.
        const bool whole = t + L <= a.T_;
#pragma unroll
        for (int q = 0; q < (L * S::CHUNKS + 31) / 32; ++q) {
          constexpr int ROWS = 32 / S::CHUNKS;
          const int i = q * ROWS + own_row;
          const long long back = whole ? q * ROWS : (long long)min(t + i, a.T_ - 1) - (t + own_row);
          if (copies) {
            unsigned char* to = to_stage + i * S::ROW + own_c * sizeof(T);
            cp_async16(to, qx + back * a.xt);
            cp_async16(to + S::ARRAY, qd + back * a.dtt);
            if (gated) cp_async16(to + 2 * S::ARRAY, qz + back * a.zt);
          }
        }
        for (int k = 0; k < NB; ++k) {
#pragma unroll
          for (int q = 0; q < L * PER / 32; ++q) {
            const int i = q * (32 / PER) + v_row;
            const long long back = whole ? q * (32 / PER) : (long long)min(t + i, a.T_ - 1) - (t + v_row);
            if (k * 16 + v_c % 16 < a.N && (!ENDS || v_c < 16))
              cp_async16(to_stage + 3 * S::ARRAY + ((k * L + i) * 32 + v_c) * sizeof(T), qv + back * qs + k * 16);
          }
        }
        qx += L * a.xt, qd += L * a.dtt, qv += L * qs;
        if (gated) qz += L * a.zt;
      }
    }
    cp_async_commit();
  };
  const auto put = [&](int stage) {
    if constexpr (EDGE) {
      unsigned char* to_stage = ring + stage * stage_bytes;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        typename S::Raw* to = (typename S::Raw*)(to_stage + (ln + r * LN) * S::ROW) + lane / LN;
        to[0] = ex[r];
        to[S::ARRAY / sizeof(typename S::Raw)] = ed[r];
        to[2 * S::ARRAY / sizeof(typename S::Raw)] = ez[r];
      }
      if constexpr (ONE) {
#pragma unroll
        for (int i = 0; i < L; ++i) ((T*)(to_stage + 3 * S::ARRAY))[i * 32 + lane] = n < a.N ? ev[i] : narrow<T>(0.f);
      }
    }
  };
  if constexpr (!EDGE) {  // states past the last stay zero
    for (int k = lane; k < S::STAGES * stage_bytes / 16; k += 32) ((float4*)ring)[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncwarp();
  }
  const auto finish = [&](float2 x, float2 z, float2 y, bool gate, bool there) {
    float2 v = fma2(skip, x, y);
    if (gate) v = mul2(v, mul2(z, sigmoid<T>(z)));
    P::store(py, there ? at.count : 0, v);
    py += LN * a.yt;
  };
  // Each lane the starts of one of the next 32 tiles, a bit a token.
  const auto flags = [&](int t) {
    unsigned f = 0;
    if (ps) {
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const int u = t + lane * L + i;
        if (u < at.t1 && ps[u]) f |= 1u << i;
      }
    }
    return f;
  };

  unsigned flag = 0, dropped = 0;
#pragma unroll
  for (int k = 0; k < S::STAGES - 1; ++k) {
    get(at.t0 + k * L, k);
    put(k);
  }
  int stage = 0;
  for (int t = at.t0; t < at.t1; t += L) {
    const int number = (t - at.t0) / L % 32;
    if (number == 0) flag = flags(t);
    const unsigned starts = __shfl_sync(0xffffffffu, flag, number);
    dropped |= starts;
    cp_async_wait<S::STAGES - 2>();
    __syncwarp();  // the tile is there, and the one before it is done with
    const int fill = stage == 0 ? S::STAGES - 1 : stage - 1;
    get(t + (S::STAGES - 1) * L, fill);
    const unsigned char* tile = ring + stage * stage_bytes;
    const auto pair = [&](int array, int r) {
      return P::wide(((const typename S::Raw*)(tile + array * S::ARRAY + (ln + r * LN) * S::ROW))[lane / LN]);
    };
    // B and C of the tile, widened.
    if constexpr (EDGE && !ONE) {
      for (int k = 0; k < NB; ++k) {
#pragma unroll
        for (int i = 0; i < L; ++i) {
          const int s = k * 16 + n;
          vs[(k * L + i) * 32 + lane] = s < a.N ? widen(pv[(long long)min(t + i, a.T_ - 1) * sv + s]) : 0.f;
        }
      }
    } else {
      for (int k = 0; k < NB; ++k) {
#pragma unroll
        for (int q = 0; q < L / V; ++q) {
          const int c = k * L * 32 + (q * 32 + lane) * V;
          float f[V];
          widen_pack(ld_pack<T, V>((const T*)(tile + 3 * S::ARRAY) + c), f);
#pragma unroll
          for (int e = 0; e < V; e += 4) *(float4*)(vs + c + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
        }
      }
    }
    float2 d[R], y[ONE ? 1 : R];  // of the lane's own tokens
    const auto sizes = [&](auto soft) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        d[r] = add2(pair(1, r), bias);
        if constexpr (decltype(soft)::value) d[r] = softplus2<T>(d[r]);
      }
    };
    if (a.softplus) sizes(std::true_type());
    else sizes(std::false_type());
    const bool whole = t + L <= a.T_;
    if (!whole) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (t + ln + r * LN >= a.T_) d[r] = zero;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float2 u = mul2(d[r], pair(0, r));
      ds[(ln + r * LN) * (32 / LN) + lane / LN] = make_float4(d[r].x, d[r].y, u.x, u.y);
      if constexpr (ENDS) sum = add2(sum, d[r]);
      if constexpr (!ONE) y[r] = zero;
    }
    __syncwarp();

    for (int k = 0; k < NB; ++k) {
      if constexpr (!ONE) {
        rates(k);
        get_h(k);
      }
      if (!ENDS && a.kept && t % kSscTile == 0)
        ssc_store_any<M>(a.vec, a.kept + ((at.b * a.tiles + t / kSscTile) * a.D + at.ch) * a.N, k * 16 + ln * M, a.N, at.count, h);
      // A whole tile without starts has no branch between its tokens, so that their instructions mix.
      const auto tokens = [&](auto plain, auto with_gate) {
        constexpr bool STARTS = !decltype(plain)::value, GATE = decltype(with_gate)::value;
        float2 held[LN];  // the lane's part of the last LN tokens' sums
#pragma unroll
        for (int i = 0; i < L; ++i) {
          const int r = i / LN, q = i % LN;
          const float4 du = ds[i * (32 / LN) + lane / LN];
          if (STARTS && (starts >> i & 1)) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int j = 0; j < M / 2; ++j) h[c][j] = zero;
          }
          const float4* pbv = (const float4*)(vs + (k * L + i) * 32 + ln * M);
          const float2 d2[2] = {make_float2(du.x, du.x), make_float2(du.y, du.y)};
          const float2 u2[2] = {make_float2(du.z, du.z), make_float2(du.w, du.w)};
          float2 acc[2] = {zero, zero};
#pragma unroll
          for (int j = 0; j < M / 4; ++j) {
            const float4 bv = pbv[j];
            const float2 b2[2] = {make_float2(bv.x, bv.y), make_float2(bv.z, bv.w)};
            float2 c2[2];
            if constexpr (!ENDS) {
              const float4 cv = pbv[4 + j];
              c2[0] = make_float2(cv.x, cv.y), c2[1] = make_float2(cv.z, cv.w);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                float2& hh = h[c][2 * j + m];
                hh = ssc_fma(ssc_decay(rate[c][2 * j + m], d2[c]), hh, mul2(u2[c], b2[m]));
                if constexpr (!ENDS) acc[c] = ssc_fma(hh, c2[m], acc[c]);
              }
            }
          }
          if constexpr (!ENDS) {
            held[q] = make_float2(acc[0].x + acc[0].y, acc[1].x + acc[1].y);
            if (q == LN - 1) {  // over the lanes: each ends with the sum of its own token
#pragma unroll
              for (int bit = 1; bit < LN; bit *= 2) {
                const bool up = ln & bit;
#pragma unroll
                for (int p = 0; p < LN / (2 * bit); ++p) {
                  const float2 send = up ? held[2 * p] : held[2 * p + 1], keep = up ? held[2 * p + 1] : held[2 * p];
                  held[p] = add2(keep, make_float2(__shfl_xor_sync(0xffffffffu, send.x, bit), __shfl_xor_sync(0xffffffffu, send.y, bit)));
                }
              }
              if constexpr (ONE) {
                if constexpr (STARTS) finish(pair(0, r), gated ? pair(2, r) : zero, held[0], gated, t + ln + r * LN < a.T_);
                else finish(pair(0, r), GATE ? pair(2, r) : zero, held[0], GATE, true);
              } else {
                y[r] = add2(y[r], held[0]);
              }
            }
          }
        }
      };
      if (starts || !whole) tokens(std::false_type(), std::false_type());
      else if (gated) tokens(std::true_type(), std::true_type());
      else tokens(std::true_type(), std::false_type());
      if constexpr (!ONE) put_h(k);
    }
    if constexpr (!ONE && !ENDS) {
#pragma unroll
      for (int r = 0; r < R; ++r) finish(pair(0, r), gated ? pair(2, r) : zero, y[r], gated, t + ln + r * LN < a.T_);
    }
    put(fill);
    stage = stage == S::STAGES - 1 ? 0 : stage + 1;
  }

  float* out = nullptr;
  if constexpr (ENDS) {
    const long long pr = at.b * (a.parts - 1) + at.part;
    out = a.ends + (pr * a.D + at.ch) * a.N;
#pragma unroll
    for (int bit = 1; bit < LN; bit *= 2)
      sum = add2(sum, make_float2(__shfl_xor_sync(0xffffffffu, sum.x, bit), __shfl_xor_sync(0xffffffffu, sum.y, bit)));
    if (ln == 0) {
      if (at.count > 0) a.sums[pr * a.D + at.ch] = sum.x;
      if (at.count > 1) a.sums[pr * a.D + at.ch + 1] = sum.y;
    }
    if (lane == 0 && at.ch == 0) a.drops[pr] = dropped ? 1.f : 0.f;
  } else {
    if (a.last && at.part == a.parts - 1) out = a.last + row * a.N;
  }
  if (out) {
    for (int k = 0; k < NB; ++k) {
      if constexpr (!ONE) get_h(k);
      ssc_store_any<M>(a.vec, out, k * 16 + ln * M, a.N, at.count, h);
    }
  }
}

// What each part but the first passes back of a carry of zero, and its sum of D: only C, e and
// the decays are needed.
template <class T, bool EDGE, bool ONE>
__global__ void __launch_bounds__(kSscThreads, 4) ssc_carry_kernel(const __grid_constant__ SscArgs<T> a) {
  pdl_entry();
  const int NP = ONE ? 16 : a.NP;
  extern __shared__ __align__(16) float2 ssc_shared[];
  float2* ds = ssc_shared;
  float2* es = ssc_shared + SscShared::kDx;
  float2* cs = es + SscShared::kE;
  float2* gs = cs + kSscTile * NP;
  float2* sums = gs + (ONE ? 0 : NP / 16 * 4 * kSscThreads);
  using P = SscPair<T, EDGE>;
  const SscPlace<T> at(a, 1, a.parts - 1);
  const int NB = NP / 16;
  const float2 zero = make_float2(0.f, 0.f);
  float2 rate[4], g[4];
  if constexpr (ONE) ssc_rates(a, at, 0, rate);
#pragma unroll
  for (int s = 0; s < 4; ++s) g[s] = zero;
  if constexpr (!ONE) {
    for (int k = 0; k < NB * 4; ++k) gs[k * kSscThreads + threadIdx.x] = zero;
  }
  float2 bias = zero, sum = zero;
  if (a.bias) bias = make_float2(at.count > 0 ? a.bias[at.ch] : 0.f, at.count > 1 ? a.bias[at.ch + 1] : 0.f);
  const int own = at.warp * kSscRows;
  unsigned dropped = 0;
  for (int tile = at.tile1 - 1; tile >= at.tile0; --tile) {
    const int t0 = tile * kSscTile;
    const long long tr = (long long)t0 + own;
    const T* pdt = a.dt + at.b * a.dtb + tr * a.dtt + at.ch;
    const T* pdy = a.dy + at.b * a.dyb + tr * a.dyt + at.ch;
    const T* pz = a.z ? a.z + at.b * a.zb + tr * a.zt + at.ch : nullptr;
    typename P::Raw dt[kSscRows], dy[kSscRows], z[kSscRows];
#pragma unroll
    for (int i = 0; i < kSscRows; ++i) {
      const int count = t0 + own + i < a.T_ ? at.count : 0;
      dt[i] = P::load(pdt + i * a.dtt, count);
      dy[i] = P::load(pdy + i * a.dyt, count);
      if (pz) z[i] = P::load(pz + i * a.zt, count);
    }
    const unsigned starts = ssc_starts(a, at.b, t0, at.lane);
    dropped |= starts;
    ssc_vectors(a, a.c + at.b * a.cb + (long long)t0 * a.ct + at.group * a.cg, a.ct, t0, NP, cs);
#pragma unroll
    for (int i = 0; i < kSscRows; ++i) {
      float2 d = ssc_step_size(a, add2(P::wide(dt[i]), bias)), e = P::wide(dy[i]);
      if (t0 + own + i >= a.T_) d = zero;
      if (pz) {
        const float2 zv = P::wide(z[i]);
        e = mul2(e, mul2(zv, sigmoid<T>(zv)));
      }
      ds[(own + i) * 32 + at.lane] = d;
      es[(own + i) * 32 + at.lane] = e;
      sum = add2(sum, d);
    }
    __syncthreads();
    for (int k = 0; k < NB; ++k) {
      if constexpr (!ONE) {
        ssc_rates(a, at, k * 16, rate);
#pragma unroll
        for (int s = 0; s < 4; ++s) g[s] = gs[(k * 4 + s) * kSscThreads + threadIdx.x];
      }
#pragma unroll 4
      for (int t = kSscTile - 1; t >= 0; --t) {
        const float2 d = ds[t * 32 + at.pr], e = es[t * 32 + at.pr];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 cv = *(const float4*)(cs + t * NP + ssc_state(k * 16, at.ln, 2 * j));
          g[2 * j] = mul2(ssc_decay(rate[2 * j], d), fma2(e, make_float2(cv.x, cv.y), g[2 * j]));
          g[2 * j + 1] = mul2(ssc_decay(rate[2 * j + 1], d), fma2(e, make_float2(cv.z, cv.w), g[2 * j + 1]));
        }
        if (starts >> t & 1) {
#pragma unroll
          for (int s = 0; s < 4; ++s) g[s] = zero;
        }
      }
      if constexpr (!ONE) {
#pragma unroll
        for (int s = 0; s < 4; ++s) gs[(k * 4 + s) * kSscThreads + threadIdx.x] = g[s];
      }
    }
    __syncthreads();
  }
  const long long row = at.b * (a.parts - 1) + at.part - 1;
  ssc_write_sums(a, at, sum, dropped != 0, row, sums);
  for (int k = 0; k < NB; ++k) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const float2 v = ONE ? g[s] : gs[(k * 4 + s) * kSscThreads + threadIdx.x];
      ssc_store(a.ends + (row * a.D + at.chb) * a.N, ssc_state(k * 16, at.ln, s), a.N, at.countb, v);
    }
  }
}

// One step of a sum over lanes that differ in bit `bit`: a lane keeps the half of its values
// that the bit names and adds its neighbour's.
template <int M> __device__ __forceinline__ void ssc_exchange(float (&v)[M], int lane, int bit) {
  const bool up = lane & bit;
#pragma unroll
  for (int k = 0; k < M / 2; ++k) {
    const float send = up ? v[k] : v[k + M / 2], keep = up ? v[k + M / 2] : v[k];
    v[k] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
  }
}

// The gradient: tiles from the last to the first.  Phase B of a tile goes forward from the kept
// state, leaving the states before tokens 4, 8 and 12 in shared memory, and then takes its four
// quarters from the last to the first: forward again with decays and states in registers, then
// backward.
template <class T, bool EDGE, bool ONE>
__global__ void __launch_bounds__(kSscThreads, 2) ssc_backward_kernel(const __grid_constant__ SscArgs<T> a) {
  pdl_entry();
  const int NP = ONE ? 16 : a.NP;
  extern __shared__ __align__(16) float2 ssc_shared[];
  float4* dxs = (float4*)ssc_shared;
  float2* es = ssc_shared + SscShared::kDx;
  float2* part = es + SscShared::kE;  // of B . g, q . A, C . h
  float2* save = part + 3 * SscShared::kPart;
  float* red = (float*)(save + SscShared::kSave);
  float2* bs = (float2*)red + SscShared::kRed;
  float2* cs = bs + kSscTile * NP;
  float2* gs = cs + kSscTile * NP;
  using P = SscPair<T, EDGE>;
  const SscPlace<T> at(a, 0, a.parts);
  const int NB = NP / 16;
  const float2 zero = make_float2(0.f, 0.f);
  float2* das = gs + NB * 4 * kSscThreads;

  float2 rate[4], g[4], da[4];
  for (int k = 0; k < NB; ++k) {
    ssc_rates(a, at, k * 16, rate);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int n = ssc_state(k * 16, at.ln, s);
      g[s] = da[s] = zero;
      if (a.dlast) g[s] = ssc_load(a.dlast + (at.b * a.D + at.chb) * a.N, n, a.N, at.countb, 0.f);
      g[s] = ssc_through(a, at, n, rate[s], g[s], a.parts - 2, a.parts - 1 - at.part, -1);
      if constexpr (!ONE) {
        gs[(k * 4 + s) * kSscThreads + threadIdx.x] = g[s];
        das[(k * 4 + s) * kSscThreads + threadIdx.x] = zero;
      }
    }
  }
  float2 bias = zero, skip = zero, dskip = zero, dbias = zero;
  if (a.bias) bias = make_float2(at.count > 0 ? a.bias[at.ch] : 0.f, at.count > 1 ? a.bias[at.ch + 1] : 0.f);
  if (a.d) skip = make_float2(at.count > 0 ? a.d[at.ch] : 0.f, at.count > 1 ? a.d[at.ch + 1] : 0.f);
  const int own = at.warp * kSscRows;
  const bool gated = a.z != nullptr;

  for (int tile = at.tile1 - 1; tile >= at.tile0; --tile) {
    const int t0 = tile * kSscTile;
    const long long tr = (long long)t0 + own;
    const T* px = a.x + at.b * a.xb + tr * a.xt + at.ch;
    const T* pdt = a.dt + at.b * a.dtb + tr * a.dtt + at.ch;
    const T* pdy = a.dy + at.b * a.dyb + tr * a.dyt + at.ch;
    const T* pz = gated ? a.z + at.b * a.zb + tr * a.zt + at.ch : nullptr;
    const unsigned starts = ssc_starts(a, at.b, t0, at.lane);
    // A
    {
      typename P::Raw x[kSscRows], dt[kSscRows], dy[kSscRows], z[kSscRows];
#pragma unroll
      for (int i = 0; i < kSscRows; ++i) {
        const int count = t0 + own + i < a.T_ ? at.count : 0;
        x[i] = P::load(px + i * a.xt, count);
        dt[i] = P::load(pdt + i * a.dtt, count);
        dy[i] = P::load(pdy + i * a.dyt, count);
        if (gated) z[i] = P::load(pz + i * a.zt, count);
      }
      ssc_vectors(a, a.b + at.b * a.bb + (long long)t0 * a.bt + at.group * a.bg, a.bt, t0, NP, bs);
      ssc_vectors(a, a.c + at.b * a.cb + (long long)t0 * a.ct + at.group * a.cg, a.ct, t0, NP, cs);
#pragma unroll
      for (int i = 0; i < kSscRows; ++i) {
        float2 d = ssc_step_size(a, add2(P::wide(dt[i]), bias)), e = P::wide(dy[i]);
        if (t0 + own + i >= a.T_) d = zero;
        const float2 u = mul2(d, P::wide(x[i]));
        if (gated) {
          const float2 zv = P::wide(z[i]);
          e = mul2(e, mul2(zv, sigmoid<T>(zv)));
        }
        dxs[(own + i) * 32 + at.lane] = make_float4(d.x, d.y, u.x, u.y);
        es[(own + i) * 32 + at.lane] = e;
      }
    }
    __syncthreads();
    // B
    for (int k = 0; k < NB; ++k) {
      if constexpr (!ONE) {
        ssc_rates(a, at, k * 16, rate);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          g[s] = gs[(k * 4 + s) * kSscThreads + threadIdx.x];
          da[s] = das[(k * 4 + s) * kSscThreads + threadIdx.x];
        }
      }
      const float* kept = a.kept + ((at.b * a.tiles + tile) * a.D + at.chb) * a.N;
      float2 h[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) h[s] = ssc_load(kept, ssc_state(k * 16, at.ln, s), a.N, at.countb, 0.f);
#pragma unroll 4
      for (int t = 0; t < 12; ++t) {
        const float4 q = dxs[t * 32 + at.pr];
        const float2 d = make_float2(q.x, q.y), u = make_float2(q.z, q.w);
        if (starts >> t & 1) {
#pragma unroll
          for (int s = 0; s < 4; ++s) h[s] = zero;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 bv = *(const float4*)(bs + t * NP + ssc_state(k * 16, at.ln, 2 * j));
          h[2 * j] = fma2(ssc_decay(rate[2 * j], d), h[2 * j], mul2(u, make_float2(bv.x, bv.y)));
          h[2 * j + 1] = fma2(ssc_decay(rate[2 * j + 1], d), h[2 * j + 1], mul2(u, make_float2(bv.z, bv.w)));
        }
        if ((t & 3) == 3) {
#pragma unroll
          for (int s = 0; s < 4; ++s) save[((t >> 2) * 4 + s) * kSscThreads + threadIdx.x] = h[s];
        }
      }
      for (int quarter = 3; quarter >= 0; --quarter) {
        float2 before[4][4], decay[4][4];  // of a token: the state that the one before it left, its decay
        if (quarter == 0) {
#pragma unroll
          for (int s = 0; s < 4; ++s) h[s] = ssc_load(kept, ssc_state(k * 16, at.ln, s), a.N, at.countb, 0.f);
        } else {
#pragma unroll
          for (int s = 0; s < 4; ++s) h[s] = save[((quarter - 1) * 4 + s) * kSscThreads + threadIdx.x];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = quarter * 4 + i;
          const float4 q = dxs[t * 32 + at.pr];
          const float2 d = make_float2(q.x, q.y), u = make_float2(q.z, q.w);
#pragma unroll
          for (int s = 0; s < 4; ++s) before[i][s] = h[s];
          if (starts >> t & 1) {
#pragma unroll
            for (int s = 0; s < 4; ++s) h[s] = zero;
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float4 bv = *(const float4*)(bs + t * NP + ssc_state(k * 16, at.ln, 2 * j));
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const int s = 2 * j + m;
              decay[i][s] = ssc_decay(rate[s], d);
              h[s] = fma2(decay[i][s], h[s], mul2(u, m ? make_float2(bv.z, bv.w) : make_float2(bv.x, bv.y)));
            }
          }
        }
#pragma unroll
        for (int i = 3; i >= 0; --i) {
          const int t = quarter * 4 + i;
          const float4 q = dxs[t * 32 + at.pr];
          const float2 d = make_float2(q.x, q.y), u = make_float2(q.z, q.w), e = es[t * 32 + at.pr];
          const bool start = starts >> t & 1;
          float2 along = zero, through = zero, y = zero;
          float v[8];  // dB and dC of the four states, summed over the pair
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float4 bv = *(const float4*)(bs + t * NP + ssc_state(k * 16, at.ln, 2 * j));
            const float4 cv = *(const float4*)(cs + t * NP + ssc_state(k * 16, at.ln, 2 * j));
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const int s = 2 * j + m;
              const float2 bb = m ? make_float2(bv.z, bv.w) : make_float2(bv.x, bv.y);
              const float2 cc = m ? make_float2(cv.z, cv.w) : make_float2(cv.x, cv.y);
              const float2 now = i == 3 ? h[s] : before[i == 3 ? 0 : i + 1][s];  // h_t
              g[s] = fma2(e, cc, g[s]);
              v[s] = fmaf(g[s].x, u.x, g[s].y * u.y);
              v[4 + s] = fmaf(e.x, now.x, e.y * now.y);
              along = fma2(g[s], bb, along);
              if (gated) y = fma2(now, cc, y);
              if (start) {
                g[s] = zero;
              } else {
                g[s] = mul2(decay[i][s], g[s]);
                const float2 qv = mul2(g[s], before[i][s]);
                through = fma2(qv, rate[s], through);
                da[s] = fma2(qv, d, da[s]);
              }
            }
          }
          if (!ONE && k > 0) {
            const int place = (t * 32 + at.pr) * 4 + ssc_half(at.pr, at.ln >> 1) * 2 + (at.ln & 1);
            along = add2(along, part[place]);
            through = add2(through, part[SscShared::kPart + place]);
            y = add2(y, part[2 * SscShared::kPart + place]);
          }
          ssc_put(part, t, at.pr, at.ln, along);
          ssc_put(part + SscShared::kPart, t, at.pr, at.ln, through);
          if (gated) ssc_put(part + 2 * SscShared::kPart, t, at.pr, at.ln, y);
          // Over the 8 pairs of the warp: the lane keeps value 4 bit2 + 2 bit3 + bit4 of its lane number.
          ssc_exchange(v, at.lane, 4);
          float v4[4] = {v[0], v[1], v[2], v[3]};
          ssc_exchange(v4, at.lane, 8);
          float v2[2] = {v4[0], v4[1]};
          ssc_exchange(v2, at.lane, 16);
          red[(t * 4 + at.warp) * 32 + at.lane] = v2[0];
        }
      }
      __syncthreads();
      // The block's sums for B and C: 16 tokens of 32 values, over the four warps.
      {
        const int which = (at.lane >> 2 & 1) * 4 + (at.lane >> 3 & 1) * 2 + (at.lane >> 4 & 1);
        const int n = ssc_state(k * 16, at.ln, which & 3);
        float* out = which < 4 ? a.part_b : a.part_c;
#pragma unroll
        for (int i = 0; i < kSscRows; ++i) {
          const int t = own + i;
          const float* r = red + t * 128 + at.lane;
          const float s = (r[0] + r[32]) + (r[64] + r[96]);
          if (n < a.N && t0 + t < a.T_)
            out[(((at.block * a.B + at.b) * a.T_ + t0 + t) * a.G + at.group) * a.N + n] = s;
        }
      }
      if constexpr (!ONE) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          gs[(k * 4 + s) * kSscThreads + threadIdx.x] = g[s];
          das[(k * 4 + s) * kSscThreads + threadIdx.x] = da[s];
        }
        if (k + 1 < NB) __syncthreads();  // before the sums are written again
      }
    }
    // C
#pragma unroll
    for (int i = 0; i < kSscRows; ++i) {
      const int count = t0 + own + i < a.T_ ? at.count : 0;
      const float2 x = P::wide(P::load(px + i * a.xt, count));
      const float4 q = dxs[(own + i) * 32 + at.lane];
      const float2 d = make_float2(q.x, q.y), e = es[(own + i) * 32 + at.lane];
      const float2 along = ssc_get(part, own + i, at.lane);
      const float2 through = mul2(ssc_get(part + SscShared::kPart, own + i, at.lane), make_float2(kLn2, kLn2));
      const float2 dx = fma2(skip, e, mul2(d, along));
      float2 dd = fma2(x, along, through);
      if (a.softplus) dd = mul2(dd, sigmoid<T>(add2(P::wide(P::load(pdt + i * a.dtt, count)), bias)));
      if (!count) dd = zero;
      dskip = fma2(e, x, dskip);
      dbias = add2(dbias, dd);
      const long long t = t0 + own + i;
      P::store(a.dx + at.b * a.dxb + t * a.dxt + at.ch, count, dx);
      P::store(a.ddt + at.b * a.ddtb + t * a.ddtt + at.ch, count, dd);
      if (gated) {
        const float2 z = P::wide(P::load(pz + i * a.zt, count)), s = sigmoid<T>(z);
        const float2 y = fma2(skip, x, ssc_get(part + 2 * SscShared::kPart, own + i, at.lane));
        const float2 slope = fma2(mul2(z, s), fma2(s, make_float2(-1.f, -1.f), make_float2(1.f, 1.f)), s);
        const float2 dy = P::wide(P::load(pdy + i * a.dyt, count));
        P::store(a.dz + at.b * a.dzb + t * a.dzt + at.ch, count, mul2(mul2(dy, y), slope));
      }
    }
  }

  // The sums over the part's tokens.
  const long long row = at.b * a.parts + at.part;
  float* pa = a.part_a + row * a.D * (a.N + 2);
  for (int k = 0; k < NB; ++k) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int n = ssc_state(k * 16, at.ln, s);
      const float2 v = ONE ? da[s] : das[(k * 4 + s) * kSscThreads + threadIdx.x];
      const float2 c = ONE ? g[s] : gs[(k * 4 + s) * kSscThreads + threadIdx.x];
      ssc_store(pa + (long long)at.chb * a.N, n, a.N, at.countb, v);
      if (a.dh0 && at.part == 0) ssc_store(a.dh0 + (at.b * a.D + at.chb) * a.N, n, a.N, at.countb, c);
    }
  }
  __syncthreads();
  part[at.warp * 32 + at.lane] = dskip;
  part[128 + at.warp * 32 + at.lane] = dbias;
  __syncthreads();
  if (at.warp < 2) {
    const float2* p = part + at.warp * 128 + at.lane;
    const float2 s = add2(add2(p[0], p[32]), add2(p[64], p[96]));
    float* out = pa + (long long)a.D * a.N + at.warp * a.D + at.ch;
    if (at.count > 0) out[0] = s.x;
    if (at.count > 1) out[1] = s.y;
  }
}

// Sums the parts in a fixed order: the blocks' of dB and dC, the rows' of dA, dd and dbias.
template <class T> struct SscFoldArgs {
  const float *part_b, *part_c, *part_a;
  T *db, *dc;
  long long dbb, dbt, dbg, dcb, dct, dcg;
  float *da, *dd, *dbias;
  long long vectors;  // B T G N
  long long vector_blocks, rows;
  int T_, D, N, G, blocks;
};
template <class T>
__global__ void __launch_bounds__(256) ssc_fold_kernel(const __grid_constant__ SscFoldArgs<T> a) {
  pdl_entry();
  if (blockIdx.x < 2 * a.vector_blocks) {
    const bool second = blockIdx.x >= a.vector_blocks;
    const long long k = (blockIdx.x - (second ? a.vector_blocks : 0)) * 256 + threadIdx.x;
    if (k >= a.vectors) return;
    const float* p = (second ? a.part_c : a.part_b) + k;
    float s = 0.f;
#pragma unroll 8
    for (int i = 0; i < a.blocks; ++i) s += p[i * a.vectors];
    long long u = k;
    const int n = (int)(u % a.N);
    u /= a.N;
    const int g = (int)(u % a.G);
    u /= a.G;
    const long long t = u % a.T_, b = u / a.T_;
    T* out = second ? a.dc + b * a.dcb + t * a.dct + g * a.dcg : a.db + b * a.dbb + t * a.dbt + g * a.dbg;
    out[n] = narrow<T>(s);
    return;
  }
  // 32 values a block; its 8 warps take every 8th row, then one warp the 8 sums.
  __shared__ float sums[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long width = (long long)a.D * (a.N + 2), at = (blockIdx.x - 2 * a.vector_blocks) * 32 + lane;
  float s = 0.f;
  if (at < width) {
#pragma unroll 8
    for (long long r = warp; r < a.rows; r += 8) s += a.part_a[r * width + at];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && at < width) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += sums[k][lane];
    const long long dn = (long long)a.D * a.N;
    if (at < dn) a.da[at] = s;
    else if (at < dn + a.D) {
      if (a.dd) a.dd[at - dn] = s;
    } else if (a.dbias) {
      a.dbias[at - dn - a.D] = s;
    }
  }
}

// ---- one token a call ------------------------------------------------------------------

template <class T> struct SscStepArgs {
  const T *x, *dt, *z, *b, *c;
  T* y;
  long long sx, sdt, sz, sy, sb, sbg, sc, scg, pool, n;  // n: channels of all rows
  const float *a, *d, *bias;
  float* state;
  const int32_t* slots;
  int D, N, DG, softplus;
  ErrSink err;
};

// Four lanes a channel, four neighbouring states a lane (VEC: as one 16-byte access).
template <class T, bool VEC>
__global__ void __launch_bounds__(128) ssc_step_kernel(const __grid_constant__ SscStepArgs<T> a) {
  pdl_entry();
  const long long at = ((long long)blockIdx.x * 128 + threadIdx.x) >> 2;
  const int ln = threadIdx.x & 3;
  const bool live = at < a.n;
  const long long b = live ? at / a.D : 0;
  const int ch = live ? (int)(at % a.D) : 0, group = ch / a.DG;
  long long slot = a.slots ? (long long)a.slots[b] : b;
  if (slot >= a.pool) {  // no such state: reported, and the row treated as padding
    if (live && ch == 0 && ln == 0) raise_err(a.err, ERRBIT_RANGE);
    slot = -1;
  }
  float y = 0.f;
  if (live && slot >= 0) {
    const float x = widen(a.x[b * a.sx + ch]);
    const float v = widen(a.dt[b * a.sdt + ch]) + (a.bias ? a.bias[ch] : 0.f);
    const float step = a.softplus ? softplus2<T>(make_float2(v, v)).x : v;
    const T *pb = a.b + b * a.sb + group * a.sbg, *pc = a.c + b * a.sc + group * a.scg;
    float* ps = a.state + (slot * a.D + ch) * a.N;
    const float* pa = a.a + (long long)ch * a.N;
    for (int n0 = ln * 4; n0 < a.N; n0 += 16) {
      float h[4], r[4];
      if constexpr (VEC) {
        const float4 q = *(const float4*)(ps + n0), w = *(const float4*)(pa + n0);
        h[0] = q.x, h[1] = q.y, h[2] = q.z, h[3] = q.w;
        r[0] = w.x, r[1] = w.y, r[2] = w.z, r[3] = w.w;
      } else {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          h[s] = n0 + s < a.N ? ps[n0 + s] : 0.f;
          r[s] = n0 + s < a.N ? pa[n0 + s] : 0.f;
        }
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (VEC || n0 + s < a.N) {
          h[s] = fmaf(ex2(step * (r[s] * kLog2e)), h[s], step * x * widen(pb[n0 + s]));
          y = fmaf(h[s], widen(pc[n0 + s]), y);
        }
      }
      if constexpr (VEC) {
        *(float4*)(ps + n0) = make_float4(h[0], h[1], h[2], h[3]);
      } else {
#pragma unroll
        for (int s = 0; s < 4; ++s)
          if (n0 + s < a.N) ps[n0 + s] = h[s];
      }
    }
    if (ln == 0 && a.d) y = fmaf(a.d[ch], x, y);
  }
  y += __shfl_xor_sync(0xffffffffu, y, 1);
  y += __shfl_xor_sync(0xffffffffu, y, 2);
  if (live && ln == 0) {
    if (slot >= 0 && a.z) {
      const float z = widen(a.z[b * a.sz + ch]);
      y *= z * sigmoid<T>(make_float2(z, z)).x;
    }
    a.y[b * a.sy + ch] = narrow<T>(y);
  }
}

// ---- launches --------------------------------------------------------------------------

// Whether every row of the array starts on a boundary of V values.
template <class T> bool ssc_rows(const SeqArray& s, int V, long long B, long long T_) {
  if (!s.p) return true;
  return (uintptr_t)s.p % (V * sizeof(T)) == 0 && (B <= 1 || s.sb % V == 0) && (T_ <= 1 || s.st % V == 0);
}
template <class T> bool ssc_rows(const GroupArray& s, int V, long long B, long long T_, long long G) {
  return (uintptr_t)s.p % (V * sizeof(T)) == 0 && (B <= 1 || s.sb % V == 0) && (T_ <= 1 || s.st % V == 0) &&
         (G <= 1 || s.sg % V == 0);
}

template <class T> SscArgs<T> ssc_args(const SelectiveScanJob& j, const SscSplit& split) {
  SscArgs<T> a = {};
  a.x = (const T*)j.x.p, a.xb = j.x.sb, a.xt = j.x.st;
  a.dt = (const T*)j.dt.p, a.dtb = j.dt.sb, a.dtt = j.dt.st;
  a.z = (const T*)j.z.p, a.zb = j.z.sb, a.zt = j.z.st;
  a.y = (T*)j.y.p, a.yb = j.y.sb, a.yt = j.y.st;
  a.b = (const T*)j.b.p, a.bb = j.b.sb, a.bt = j.b.st, a.bg = j.b.sg;
  a.c = (const T*)j.c.p, a.cb = j.c.sb, a.ct = j.c.st, a.cg = j.c.sg;
  a.dy = (const T*)j.dy.p, a.dyb = j.dy.sb, a.dyt = j.dy.st;
  a.dx = (T*)j.dx.p, a.dxb = j.dx.sb, a.dxt = j.dx.st;
  a.ddt = (T*)j.ddt.p, a.ddtb = j.ddt.sb, a.ddtt = j.ddt.st;
  a.dz = (T*)j.dz.p, a.dzb = j.dz.sb, a.dzt = j.dz.st;
  a.a = j.a, a.d = j.d, a.bias = j.bias, a.h0 = j.h0, a.dlast = j.dlast, a.starts = j.starts;
  a.last = j.last, a.kept = j.kept, a.dh0 = j.dh0;
  a.B = j.B, a.T_ = (int)j.T, a.D = (int)j.D, a.N = (int)j.N, a.NP = (int)((j.N + 15) / 16 * 16);
  a.G = (int)j.G, a.DG = (int)(j.D / j.G), a.blocks = (a.DG + kSscChannels - 1) / kSscChannels;
  a.tiles = (int)((j.T + kSscTile - 1) / kSscTile);
  a.parts = (int)split.parts, a.part_tiles = (int)split.tiles, a.softplus = j.softplus;
  a.vec = j.N % 4 == 0;
  for (const void* q : {(const void*)j.a, (const void*)j.h0, (const void*)j.last, (const void*)j.kept}) a.vec = a.vec && (uintptr_t)q % 16 == 0;
  float* p = (float*)j.temp;
  a.ends = p;
  a.sums = a.ends + j.B * (split.parts - 1) * j.D * j.N;
  a.drops = a.sums + j.B * (split.parts - 1) * j.D;
  a.part_a = a.drops + j.B * (split.parts - 1);
  a.part_b = a.part_a + j.B * split.parts * j.D * (j.N + 2);
  a.part_c = a.part_b + (long long)a.blocks * j.B * j.T * j.G * j.N;
  return a;
}

template <class K, class A> cudaError_t ssc_launch(K kernel, long long grid, size_t smem, const A& a, const LaunchCtx& ctx) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, (unsigned)grid, kSscThreads, smem, ctx.stream, a);
}

template <class T, bool EDGE, bool ONE, int LN> cudaError_t ssc_forward(const SelectiveScanJob& j, const SscForwardPlan& plan, const LaunchCtx& ctx) {
  const SscArgs<T> a = ssc_args<T>(j, plan.split);
  const long long units = j.B * a.G * ((a.DG + 64 / LN - 1) / (64 / LN));
  const auto grid = [&](long long parts) { return (units * parts + kSscThreads / 32 - 1) / (kSscThreads / 32); };
  using S = SscLane<T, EDGE, LN>;
  const int NB = ONE ? 1 : a.NP / 16;
  const size_t smem = (size_t)(kSscThreads / 32) * S::warp_bytes(NB);
  profile_before(ctx);
  cudaError_t e = cudaSuccess;
  if (plan.split.parts > 1) e = ssc_launch(ssc_forward_kernel<T, EDGE, ONE, true, LN>, grid(plan.split.parts - 1), smem, a, ctx);
  if (e == cudaSuccess) e = ssc_launch(ssc_forward_kernel<T, EDGE, ONE, false, LN>, grid(plan.split.parts), smem, a, ctx);
  profile_after(ctx);
  return e;
}

template <class T, bool EDGE, bool ONE> cudaError_t ssc_backward(const SelectiveScanJob& j, const LaunchCtx& ctx) {
  const SscSplit split = ssc_split(j.B, j.T, j.D, j.G, true);
  const SscArgs<T> a = ssc_args<T>(j, split);
  const long long units = j.B * a.G * a.blocks;
  profile_before(ctx);
  cudaError_t e = cudaSuccess;
  if (split.parts > 1)
    e = ssc_launch(ssc_carry_kernel<T, EDGE, ONE>, units * (split.parts - 1), SscShared::carry(a.NP), a, ctx);
  if (e == cudaSuccess)
    e = ssc_launch(ssc_backward_kernel<T, EDGE, ONE>, units * split.parts, SscShared::backward(a.NP), a, ctx);
  if (e == cudaSuccess) {
    SscFoldArgs<T> f = {};
    f.part_a = a.part_a, f.part_b = a.part_b, f.part_c = a.part_c;
    f.db = (T*)j.db.p, f.dbb = j.db.sb, f.dbt = j.db.st, f.dbg = j.db.sg;
    f.dc = (T*)j.dc.p, f.dcb = j.dc.sb, f.dct = j.dc.st, f.dcg = j.dc.sg;
    f.da = j.da, f.dd = j.dd, f.dbias = j.dbias;
    f.vectors = j.B * j.T * j.G * j.N;
    f.vector_blocks = (f.vectors + 255) / 256;
    f.rows = j.B * split.parts;
    f.T_ = a.T_, f.D = a.D, f.N = a.N, f.G = a.G, f.blocks = a.blocks;
    const long long grid = 2 * f.vector_blocks + (j.D * (j.N + 2) + 31) / 32;
    e = launch_pdl(ssc_fold_kernel<T>, (unsigned)grid, 256, 0, ctx.stream, f);
  }
  profile_after(ctx);
  return e;
}

template <class T, bool EDGE> cudaError_t ssc_forward_any(const SelectiveScanJob& j, const LaunchCtx& ctx) {
  const SscForwardPlan plan = ssc_forward_plan(j.B, j.T, j.D, j.G);
  if (j.N > 16) return ssc_forward<T, EDGE, false, 4>(j, plan, ctx);
  return plan.lanes == 2 ? ssc_forward<T, EDGE, true, 2>(j, plan, ctx) : ssc_forward<T, EDGE, true, 4>(j, plan, ctx);
}
template <class T> cudaError_t launch_selective_scan(const SelectiveScanJob& j, const LaunchCtx& ctx) {
  constexpr int V = 16 / sizeof(T);
  bool even = (j.D / j.G) % V == 0 && j.N % V == 0 && ssc_rows<T>(j.b, V, j.B, j.T, j.G) && ssc_rows<T>(j.c, V, j.B, j.T, j.G);
  for (const SeqArray* s : {&j.x, &j.dt, &j.z, &j.y}) even = even && ssc_rows<T>(*s, V, j.B, j.T);
  return even ? ssc_forward_any<T, false>(j, ctx) : ssc_forward_any<T, true>(j, ctx);
}

template <class T> cudaError_t launch_selective_scan_backward(const SelectiveScanJob& j, const LaunchCtx& ctx) {
  bool even = (j.D / j.G) % 2 == 0;
  for (const SeqArray* s : {&j.x, &j.dt, &j.z, &j.dy, &j.dx, &j.ddt, &j.dz}) even = even && ssc_rows<T>(*s, 2, j.B, j.T);
  if (j.N <= 16) return even ? ssc_backward<T, false, true>(j, ctx) : ssc_backward<T, true, true>(j, ctx);
  return even ? ssc_backward<T, false, false>(j, ctx) : ssc_backward<T, true, false>(j, ctx);
}

template <class T> cudaError_t launch_selective_scan_step(const SelectiveScanStepJob& j, const LaunchCtx& ctx) {
  SscStepArgs<T> a = {};
  a.x = (const T*)j.x, a.dt = (const T*)j.dt, a.z = (const T*)j.z, a.b = (const T*)j.b, a.c = (const T*)j.c;
  a.y = (T*)j.y;
  a.sx = j.sx, a.sdt = j.sdt, a.sz = j.sz, a.sy = j.sy, a.sb = j.sb, a.sbg = j.sbg, a.sc = j.sc, a.scg = j.scg;
  a.a = j.a, a.d = j.d, a.bias = j.bias, a.state = j.state, a.slots = j.slots, a.pool = j.pool;
  a.D = (int)j.D, a.N = (int)j.N, a.DG = (int)(j.D / j.G), a.softplus = j.softplus;
  a.n = j.B * j.D;
  a.err = ctx.err;
  const bool vec = j.N % 4 == 0 && (uintptr_t)j.state % 16 == 0 && (uintptr_t)j.a % 16 == 0;
  const unsigned grid = (unsigned)((a.n + 31) / 32);
  profile_before(ctx);
  const cudaError_t e = vec ? launch_pdl(ssc_step_kernel<T, true>, grid, 128, 0, ctx.stream, a)
                            : launch_pdl(ssc_step_kernel<T, false>, grid, 128, 0, ctx.stream, a);
  profile_after(ctx);
  return e;
}

}  // namespace gbs
