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
// The gradient: a block of 4 warps takes 64 channels and tiles of 16 tokens, from the last to the
// first; a warp 16 channels, 4 lanes a pair of channels and 4 states of both a lane.  A tile's states
// are computed again from the one kept before it.  The warps meet twice a tile, for B and C and for
// the sums over channels.  Issue and shared memory bound it about equally: of some 240 instructions
// and 53 passes a token and warp, 8 passes bring D, D x, B and C forward and 6 C and e back, 12 and
// 8 instructions are the lanes' parts of the sums over states, 7 and 28 the sums over channels.
//
// The tokens of a row are one chain.  Where the rows and channels are too few for the device,
// they are split into parts: a first kernel finds what each part makes of a state of zero, and
// with exp(A sum D) each part knows where it starts (the gradient: from the other end).
//
// The states and channels of a full tile that do not exist, and its tokens behind the last, keep zeros
// beside finite inputs.  Beside an infinity they would be NaNs, so that tiles with one are gone through with
// those places put back to 0, and tokens behind the last are left out.
//
// Measured (GB300, cold caches): 8 x 2048 x 2048, 16 states, bf16, gated, with starts and kept
// states 274 us (0.7 instructions a cycle and scheduler, 0.15 of the copy rate), its gradient
// 829 us (0.56, and half of shared memory's cycles); 1 x 32768 x 2048 continued 534 us; one
// token, 64 x 4096, 17.5 us.
#pragma once

#include "lm.cuh"
#include "lm.h"

namespace gbs {

constexpr int kSscThreads = 128;

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

// How rows are read: by asynchronous copies of 16 bytes (WHOLE), of 4 (WORDS: any fp32 rows, and
// 16-bit ones with even widths, strides and counts of states on 4-byte boundaries), or value by value
// through registers (SINGLES, 16 bits only).  8 x 2048 tokens, 16 states, WORDS and SINGLES: 2046
// channels bf16 310 and 515 us, the gradient 870 and 1211; 4 x 2048 x 2001 fp32 212 and 252, 544 and 589.
enum SscMode { kSscWhole, kSscWords, kSscSingles };

// Two neighbouring channels of a row, as they lie in memory.
template <class T, SscMode MODE> struct SscPair {
  static constexpr bool EDGE = MODE == kSscSingles || (MODE == kSscWords && sizeof(T) == 4);  // not at once
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

// exp of the product, a in units of log2 e.  In single operations: a packed product before the
// exponential costs more than the instruction it saves (measured in a loop of nothing else, 32
// states a thread, 3 warps a scheduler: 6.9 cycles a state and token with packed products and sums,
// 5.2 with these and the sums single and only D x B packed, 5.9 with all of it single).
//
// The instruction's result is low by 0.3 to 0.45 units of 2^-24 on average for arguments of -0.001 to
// -0.3 (measured), which in a chain of decays adds up over as many tokens as the state lasts.  2^-25
// added to the argument leaves 0.02 to 0.1 (0.26 high below -0.001); of 0 it is 1 all the same.
// 8 x 2048 x 2048 bf16, error against 64 bits: last state 4.0e-7 without it, dA 1.2e-6.
constexpr float kSscCentre = 0x1p-25f;
__device__ __forceinline__ float2 ssc_decay(float2 a, float2 d) {
  return make_float2(ex2(fmaf(a.x, d.x, kSscCentre)), ex2(fmaf(a.y, d.y, kSscCentre)));
}
__device__ __forceinline__ float2 ssc_fma(float2 a, float2 b, float2 c) { return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)); }
// A state (or what is passed back) through a part: e is what the part makes of zero.  The part's decay, a
// product of small ones, does not go below fp32's least number: 0 times an infinite state would be a
// NaN, which no token's decay makes of it.
__device__ __forceinline__ float2 ssc_through(float2 rate, float sum, float2 h, float2 e) {
  const float2 decay = ssc_decay(rate, make_float2(sum, sum));
  return fma2(make_float2(max_nan(decay.x, 0x1p-149f), max_nan(decay.y, 0x1p-149f)), h, e);
}
// D and e go into fp32 results (states, dA, dd, dbias) whatever the inputs' type, so that their
// functions are the fp32 ones; what only 16-bit outputs see (y, dz) is as exact as their type.
template <class T> __device__ __forceinline__ float2 ssc_step_size(const SscArgs<T>& a, float2 v) {
  return a.softplus ? softplus2(v) : v;
}

// ---- forward ---------------------------------------------------------------------------

// M = 16 / LN states of two channels a thread, LN lanes a pair of channels; a warp is on its own:
// WIDTH channels, tiles of L tokens, of which a lane prepares and finishes R.  What a warp reads
// comes by asynchronous copies into a ring of STAGES tiles of its own in shared memory.
template <class T, SscMode MODE, int LN_> struct SscLane {
  static constexpr int LN = LN_, L = 8, R = L / LN, M = 16 / LN, WIDTH = 64 / LN;
  static constexpr int STAGES = sizeof(T) == 2 ? 3 : 2;
  static constexpr int ROW = WIDTH * (int)sizeof(T), ARRAY = L * ROW;  // bytes
  static constexpr int VECTORS = L * 32 * (int)sizeof(T);               // B and C of 16 states, as they are
  static constexpr int CHUNKS = ROW / 16;                               // 16-byte copies of a row
  using P = SscPair<T, MODE>;
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

// M values of two channels of a (D, N) array, in pairs of states; 0 where there are none.
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

// What a tile's tokens are gone through as: whole tiles of finite inputs without starts, with starts, any
// tile.  (8 x 2048 x 2048 bf16: starts and the rest in one loop cost the gradient 3 % more.)
enum { kSscPlain, kSscStarts, kSscAny };
template <int KIND> using SscKind = std::integral_constant<int, KIND>;

// PADDED: the states are no multiple of 16, so that tiles are looked through for infinities (8 x 2048 x 2048
// bf16, 8 states: 269 -> 276 us).  Not in ENDS, which stores nothing of the states past the last.
// ENDS: only the states that the part ends with, from a state of zero, and its sum of D.
template <class T, SscMode MODE, bool ONE, bool ENDS, bool PADDED, int LN>
__global__ void __launch_bounds__(kSscThreads, ONE && !(MODE == kSscSingles && LN == 2) ? 4 : 3) ssc_forward_kernel(const __grid_constant__ SscArgs<T> a) {
  pdl_entry();
  using S = SscLane<T, MODE, LN>;
  using P = typename S::P;
  constexpr bool SINGLES = MODE == kSscSingles;
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
  // States past the last: their b and c are 0, but 0 times an infinity is a NaN, which their c of 0
  // would bring into y.  Where an input is not finite they are put back to 0.
  const auto clear_past = [&](int k) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int j = 0; j < M / 2; ++j) {
        const int s = k * 16 + ln * M + 2 * j;
        h[c][j] = make_float2(s < a.N ? h[c][j].x : 0.f, s + 1 < a.N ? h[c][j].y : 0.f);
      }
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
            h[c][j] = dropped ? e[c][j] : ssc_through(rate[c][j], sum[c], h[c][j], e[c][j]);
      }
      if constexpr (PADDED) clear_past(k);
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

  // Starts a tile's copies into the ring.  SINGLES: loads the tile, for `put` to store behind the
  // one that is worked on.  (No ordinary load goes among the copies: waiting for it would be waiting
  // for them.)
  constexpr int V = 16 / sizeof(T), PER = 32 / V;
  const int own_row = lane / S::CHUNKS, own_c = lane % S::CHUNKS * V;   // the lane's pieces of x, dt, z
  const int v_row = lane / PER, v_c = lane % PER * V;                   // and of B or C
  const bool copies = lane < L * S::CHUNKS && own_c < at.width;
  const T* qx = px + (long long)(at.t0 + own_row) * a.xt + at.base + own_c;
  const T* qd = pdt + (long long)(at.t0 + own_row) * a.dtt + at.base + own_c;
  const T* qz = gated ? pz + (long long)(at.t0 + own_row) * a.zt + at.base + own_c : nullptr;
  const long long qs = v_c < 16 ? a.bt : a.ct;
  const T* qv = (v_c < 16 ? pb : pc) + (long long)(at.t0 + v_row) * qs + v_c % 16;
  typename S::Raw ex[SINGLES ? R : 1], ed[SINGLES ? R : 1], ez[SINGLES ? R : 1];
  T ev[SINGLES && ONE ? L : 1];
  const auto get = [&](int t, int stage) {
    unsigned char* to_stage = ring + stage * stage_bytes;
    if (t < at.t1) {
      if constexpr (SINGLES) {
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
      } else if constexpr (MODE == kSscWords) {
        constexpr int VW = 4 / sizeof(T), ROW_WORDS = 32 / VW, WORDS = S::ROW / 4;  // words of B and C, of x
        const int x_c = lane % WORDS * VW;
#pragma unroll
        for (int q = 0; q < L * WORDS / 32; ++q) {
          const int i = q * (32 / WORDS) + lane / WORDS;
          const long long row = min(t + i, a.T_ - 1);
          if (x_c < at.width) {
            unsigned char* to = to_stage + i * S::ROW + x_c * sizeof(T);
            cp_async4(to, px + row * a.xt + at.base + x_c);
            cp_async4(to + S::ARRAY, pdt + row * a.dtt + at.base + x_c);
            if (gated) cp_async4(to + 2 * S::ARRAY, pz + row * a.zt + at.base + x_c);
          }
        }
        const int w_c = lane % ROW_WORDS * VW;
        const T* from = (w_c < 16 ? pb : pc) + w_c % 16;
        for (int k = 0; k < NB; ++k) {
#pragma unroll
          for (int q = 0; q < L / VW; ++q) {
            const int i = q * VW + lane / ROW_WORDS;
            if (k * 16 + w_c % 16 < a.N && (!ENDS || w_c < 16))
              cp_async4(to_stage + 3 * S::ARRAY + ((k * L + i) * 32 + w_c) * sizeof(T),
                        from + (long long)min(t + i, a.T_ - 1) * (w_c < 16 ? a.bt : a.ct) + k * 16);
          }
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
    if constexpr (SINGLES) {
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
  if constexpr (!SINGLES) {  // states past the last, and channels, stay zero
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
    if constexpr (SINGLES && !ONE) {
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
        if constexpr (decltype(soft)::value) d[r] = softplus2(d[r]);
      }
    };
    if (a.softplus) sizes(std::true_type());
    else sizes(std::false_type());
    const bool whole = t + L <= a.T_;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 u = mul2(d[r], pair(0, r));
      if (!whole && t + ln + r * LN >= a.T_) d[r] = u = zero;  // no token
      ds[(ln + r * LN) * (32 / LN) + lane / LN] = make_float4(d[r].x, d[r].y, u.x, u.y);
      if constexpr (ENDS) sum = add2(sum, d[r]);
      if constexpr (!ONE) y[r] = zero;
    }
    bool wild = false;
    if constexpr (PADDED) {  // where D is not finite D x is not either
      float size = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 du = ds[(ln + r * LN) * (32 / LN) + lane / LN];
        size += fabsf(du.z) + fabsf(du.w);
      }
      wild = __any_sync(0xffffffffu, !(size < __int_as_float(0x7f800000)));
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
      const auto tokens = [&](auto kind, auto with_gate) {
        constexpr bool STARTS = decltype(kind)::value != kSscPlain, ANY = decltype(kind)::value == kSscAny;
        constexpr bool GATE = decltype(with_gate)::value;
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
          // Tokens behind the last are left out, since 0 times a rate or a b may be a NaN.
          if (!ANY || t + i < a.T_) {
#pragma unroll
            for (int j = 0; j < M / 4; ++j) {
              const float4 bv = pbv[j];
              const float2 b2[2] = {make_float2(bv.x, bv.y), make_float2(bv.z, bv.w)};
              float2 c2[2];
              if constexpr (!ENDS && !ANY) {
                const float4 cv = pbv[4 + j];
                c2[0] = make_float2(cv.x, cv.y), c2[1] = make_float2(cv.z, cv.w);
              }
#pragma unroll
              for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                  float2& hh = h[c][2 * j + m];
                  hh = ssc_fma(ssc_decay(rate[c][2 * j + m], d2[c]), hh, mul2(u2[c], b2[m]));
                  if constexpr (!ENDS && !ANY) acc[c] = ssc_fma(hh, c2[m], acc[c]);
                }
              }
            }
            if constexpr (!ENDS && ANY) {
              if (PADDED && wild) clear_past(k);
#pragma unroll
              for (int j = 0; j < M / 4; ++j) {
                const float4 cv = pbv[4 + j];
                const float2 c2[2] = {make_float2(cv.x, cv.y), make_float2(cv.z, cv.w)};
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                  for (int m = 0; m < 2; ++m) acc[c] = ssc_fma(h[c][2 * j + m], c2[m], acc[c]);
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
      constexpr int any = ENDS ? kSscStarts : kSscAny;  // (ENDS leaves out the last part)
      if (!whole || (PADDED && wild)) tokens(SscKind<any>(), std::false_type());
      else if (starts) tokens(SscKind<kSscStarts>(), std::false_type());
      else if (gated) tokens(SscKind<kSscPlain>(), std::true_type());
      else tokens(SscKind<kSscPlain>(), std::false_type());
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

// ---- gradient --------------------------------------------------------------------------

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

// A block takes 64 channels of a group, a warp 16 of them: 4 lanes a pair of channels, 4 states of
// both a lane.  A tile's 16 tokens go to the lanes of a pair in turn (t % 4 = ln).  In shared
// memory, for each warp: a ring of two tiles as they lie in memory; D and D x, e, of the tile;
// the lanes' parts of three sums over states for 4 tokens; states before tokens 4, 8 and 12; the
// warp's sums of dB and dC; with more than 16 states what a lane keeps of each block.  For the
// block: two tiles of B and C as they are, one widened.
template <class T, SscMode MODE> struct SscBack {
  static constexpr int L = kSscTile, R = L / 4, M = 4, STAGES = 2;
  static constexpr int ROW = 16 * (int)sizeof(T), ARRAY = L * ROW, KEPT = 16 * 16 * 4, STAGE = 4 * ARRAY + KEPT;
  static constexpr int CHUNKS = ROW / 16;
  static constexpr int DU = L * 8 * 16, E = L * 8 * 8, SUMS = 3 * 4 * 8 * 4 * 8, SAVE = 3 * 8 * 32 * 4, RED = L * 32 * 4;
  static constexpr int VECTORS = L * 32 * (int)sizeof(T);
  using P = SscPair<T, MODE>;
  using Raw = typename P::Raw;
  static __host__ __device__ constexpr int warp_bytes(int NB, bool carry) {
    return STAGES * STAGE + DU + E + (carry ? 0 : SUMS + SAVE + RED) + (NB > 1 ? NB * 2 * 8 * 32 * 4 : 0);
  }
  static __host__ __device__ constexpr int bytes(int NB, bool carry) {
    return 4 * warp_bytes(NB, carry) + STAGES * VECTORS + NB * L * 32 * 4;
  }
};

// Place of lane ln's part of token i's sums for a pair, so that neither the writes (all lanes one
// token) nor the reads (a lane its own token's four parts, 16 bytes at a time) meet in a bank.
__device__ __forceinline__ int ssc_sum_half(int i, int pair, int half) {
  const int px = pair ^ (2 * i);
  return ((i * 8 + px) * 2 + (half ^ (px >> 2 & 1))) * 2;
}

// CARRY: only what each part but the first passes back of a carry of zero, and its sum of D.
//
// Tiles go from the last to the first.  A: the lane's own tokens' D, D x, e.  B: forward from the
// kept state, leaving the states before tokens 4, 8 and 12; then the four quarters from the last to
// the first: forward again with decays and states in registers, then backward.  C, after each
// quarter: the lane's own token, from the sums over states.  The sums over channels for dB and
// dC: over the pair in the thread, over the warp by exchanges, over the block in shared memory,
// and over the blocks by a second kernel.
template <class T, SscMode MODE, bool ONE, bool CARRY>
__global__ void __launch_bounds__(kSscThreads, 2) ssc_backward_kernel(const __grid_constant__ SscArgs<T> a) {
  pdl_entry();
  using S = SscBack<T, MODE>;
  using P = typename S::P;
  constexpr bool SINGLES = MODE == kSscSingles;
  using Raw = typename S::Raw;
  constexpr int L = S::L, R = S::R, M = S::M;
  extern __shared__ __align__(16) float2 ssc_shared[];
  const int NB = ONE ? 1 : a.NP / 16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ln = lane & 3, pr = lane >> 2;
  unsigned char* ring = (unsigned char*)ssc_shared + warp * S::warp_bytes(NB, CARRY);
  float4* du = (float4*)(ring + S::STAGES * S::STAGE);  // D and D x (token, pair)
  float2* es = (float2*)(du + L * 8);                   // (token, pair)
  float2* sums = es + L * 8;                            // of B . g, q . A, C . h (which, token of 4, pair, lane)
  float4* save = (float4*)(sums + (CARRY ? 0 : 3 * 4 * 8 * 4));
  float* red = (float*)save + (CARRY ? 0 : 3 * 8 * 32);  // dB and dC over the warp (token, 32)
  float4* keep = (float4*)(red + (CARRY ? 0 : L * 32));  // g and dA by block, where there are several
  unsigned char* vring = (unsigned char*)ssc_shared + 4 * S::warp_bytes(NB, CARRY);
  float* vs = (float*)(vring + S::STAGES * S::VECTORS);  // B (16) and C (16) (block, token)
  const float2 zero = make_float2(0.f, 0.f);

  // Where the block works.
  long long unit = blockIdx.x;
  const int block = (int)(unit % a.blocks);
  unit /= a.blocks;
  const int group = (int)(unit % a.G);
  unit /= a.G;
  const int parts = CARRY ? a.parts - 1 : a.parts, part = (int)(unit % parts) + (CARRY ? 1 : 0);
  const long long b = unit / parts;
  const int tile0 = part * a.part_tiles, tile1 = min(a.tiles, tile0 + a.part_tiles);
  const int first = group * a.DG + block * kSscChannels, width = min(16, (group + 1) * a.DG - first - 16 * warp);
  const int base = width > 0 ? first + 16 * warp : first;  // a warp without channels reads real ones and stores nothing
  const int count = min(2, width - 2 * pr), ch = count > 0 ? base + 2 * pr : base;
  const long long row = b * a.D + ch;

  float2 rate[2][2], g[2][2], da[2][2], da_few[2][2];  // (channel, pair of states)
  const auto rates = [&](int k) {
    ssc_load_any<M>(a.vec, a.a + (long long)ch * a.N, k * 16 + ln * M, a.N, count, rate);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int j = 0; j < 2; ++j) rate[c][j] = mul2(rate[c][j], make_float2(kLog2e, kLog2e));
  };
  // States and channels past the last: 0 times an infinity is a NaN, which the sums over states and over
  // channels would take.  Where an input is not finite, what belongs to them is put back to 0.
  const bool padded = a.N != a.NP, special = padded || (group + 1) * a.DG - first < kSscChannels;
  const auto clear_past = [&](int k, float2 (&v)[2][2]) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int s = k * 16 + ln * M + 2 * j;
        v[c][j] = make_float2(c < count && s < a.N ? v[c][j].x : 0.f, c < count && s + 1 < a.N ? v[c][j].y : 0.f);
      }
  };
  const auto put = [&](int at, const float2 (&v)[2][2]) {
#pragma unroll
    for (int c = 0; c < 2; ++c) keep[(at * 2 + c) * 32 + lane] = make_float4(v[c][0].x, v[c][0].y, v[c][1].x, v[c][1].y);
  };
  const auto get = [&](int at, float2 (&v)[2][2]) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float4 q = keep[(at * 2 + c) * 32 + lane];
      v[c][0] = make_float2(q.x, q.y), v[c][1] = make_float2(q.z, q.w);
    }
  };
  for (int k = 0; k < NB; ++k) {
    rates(k);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int j = 0; j < 2; ++j) g[c][j] = da[c][j] = da_few[c][j] = zero;
    if constexpr (!CARRY) {
      if (a.dlast) ssc_load_any<M>(a.vec, a.dlast + row * a.N, k * 16 + ln * M, a.N, count, g);
      // Through the parts behind this one in turn.
      for (int p = a.parts - 2; p >= part; --p) {
        const long long q = b * (a.parts - 1) + p;
        float2 e[2][2];
        ssc_load_any<M>(a.vec, a.ends + (q * a.D + ch) * a.N, k * 16 + ln * M, a.N, count, e);
        const float* sp = a.sums + q * a.D + ch;
        const float sum[2] = {count > 0 ? sp[0] : 0.f, count > 1 ? sp[1] : 0.f};
        const bool dropped = a.drops[q] != 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            g[c][j] = dropped ? e[c][j] : ssc_through(rate[c][j], sum[c], g[c][j], e[c][j]);
      }
      if (padded) clear_past(k, g);
    }
    if constexpr (!ONE) {
      put(2 * k, g);
      put(2 * k + 1, da);
    }
  }
  float2 bias = zero, skip = zero, dskip = zero, dbias = zero, dskip_few = zero, dbias_few = zero, sum_d = zero;
  if (a.bias) bias = make_float2(count > 0 ? a.bias[ch] : 0.f, count > 1 ? a.bias[ch + 1] : 0.f);
  if (!CARRY && a.d) skip = make_float2(count > 0 ? a.d[ch] : 0.f, count > 1 ? a.d[ch + 1] : 0.f);
  const bool gated = a.z != nullptr;
  const T* px = a.x + b * a.xb;
  const T* pdt = a.dt + b * a.dtb;
  const T* pdy = a.dy + b * a.dyb;
  const T* pz = gated ? a.z + b * a.zb : nullptr;
  const T* pb = a.b + b * a.bb + group * a.bg;
  const T* pc = a.c + b * a.cb + group * a.cg;
  const uint8_t* ps = a.starts ? a.starts + b * a.T_ : nullptr;

  // Each lane the starts of one of the next 32 tiles, a bit a token.
  const auto flags = [&](int tile) {
    unsigned f = 0;
    const int t = (tile - lane) * L;
    if (ps && tile - lane >= tile0) {
#pragma unroll
      for (int i = 0; i < L; ++i)
        if (t + i < a.T_ && ps[t + i]) f |= 1u << i;
    }
    return f;
  };
  // Starts a tile's copies into the ring.  SINGLES: loads the tile, for `land` to store behind the
  // one that is worked on.
  constexpr int V = 16 / sizeof(T), PER = 32 / V;
  Raw ex[SINGLES ? R : 1], ed[SINGLES ? R : 1], ey[SINGLES ? R : 1], ez[SINGLES ? R : 1];
  T ev[SINGLES && ONE ? 4 : 1];
  float2 ek[2][2];
  const auto fetch = [&](int tile, int stage) {
    unsigned char* to = ring + stage * S::STAGE;
    if (tile >= tile0) {
      const int t = tile * L;
      if constexpr (SINGLES) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const long long u = min(t + 4 * r + ln, a.T_ - 1);
          if (!CARRY) ex[r] = P::load(px + u * a.xt + ch, count);
          ed[r] = P::load(pdt + u * a.dtt + ch, count);
          ey[r] = P::load(pdy + u * a.dyt + ch, count);
          if (gated) ez[r] = P::load(pz + u * a.zt + ch, count);
        }
        if constexpr (ONE) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const long long u = min(t + 4 * warp + i, a.T_ - 1);
            const int n = lane % 16 < a.N ? lane % 16 : 0;
            ev[i] = lane < 16 ? pb[u * a.bt + n] : pc[u * a.ct + n];
          }
          if constexpr (!CARRY) ssc_load_any<M>(a.vec, a.kept + ((b * a.tiles + tile) * a.D + ch) * a.N, ln * M, a.N, count, ek);
        }
      } else if constexpr (MODE == kSscWords) {
        constexpr int VW = 4 / sizeof(T), ROW_WORDS = 32 / VW, WORDS = S::ROW / 4;  // words of B and C, of x
        const int x_c = lane % WORDS * VW;
#pragma unroll
        for (int q = 0; q < L * WORDS / 32; ++q) {
          const int i = q * (32 / WORDS) + lane / WORDS;
          if (x_c < width) {
            const long long u = min(t + i, a.T_ - 1);
            unsigned char* at = to + i * S::ROW + x_c * sizeof(T);
            if (!CARRY) cp_async4(at, px + u * a.xt + base + x_c);
            cp_async4(at + S::ARRAY, pdt + u * a.dtt + base + x_c);
            cp_async4(at + 2 * S::ARRAY, pdy + u * a.dyt + base + x_c);
            if (gated) cp_async4(at + 3 * S::ARRAY, pz + u * a.zt + base + x_c);
          }
        }
        if constexpr (ONE) {
          if constexpr (!CARRY) {  // the lane's own states
            const float* from = a.kept + ((b * a.tiles + tile) * a.D + ch) * a.N + ln * M;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              unsigned char* at = to + 4 * S::ARRAY + (c * 32 + lane) * 16;
              if (a.vec) {
                if (c < count && ln * M < a.N) cp_async16(at, from + c * a.N);
              } else {
#pragma unroll
                for (int m = 0; m < M; ++m)
                  if (c < count && ln * M + m < a.N) cp_async4(at + 4 * m, from + c * a.N + m);
              }
            }
          }
          const int c = lane % ROW_WORDS * VW;
#pragma unroll
          for (int q = 0; q < 4 / VW; ++q) {
            const int i = warp * 4 + q * VW + lane / ROW_WORDS;
            const long long u = min(t + i, a.T_ - 1);
            if (c % 16 < a.N && (!CARRY || c >= 16))
              cp_async4(vring + stage * S::VECTORS + (i * 32 + c) * sizeof(T), c < 16 ? pb + u * a.bt + c : pc + u * a.ct + c - 16);
          }
        }
      } else {
#pragma unroll
        for (int q = 0; q < L * S::CHUNKS / 32; ++q) {
          const int k = q * 32 + lane, i = k / S::CHUNKS, c = k % S::CHUNKS * V;
          if (c < width) {
            const long long u = min(t + i, a.T_ - 1);
            unsigned char* at = to + i * S::ROW + c * sizeof(T);
            if (!CARRY) cp_async16(at, px + u * a.xt + base + c);
            cp_async16(at + S::ARRAY, pdt + u * a.dtt + base + c);
            cp_async16(at + 2 * S::ARRAY, pdy + u * a.dyt + base + c);
            if (gated) cp_async16(at + 3 * S::ARRAY, pz + u * a.zt + base + c);
          }
        }
        if constexpr (ONE) {
          if (!CARRY && ln * M < a.N) {  // the lane's own states
            const float* from = a.kept + ((b * a.tiles + tile) * a.D + ch) * a.N + ln * M;
#pragma unroll
            for (int c = 0; c < 2; ++c)
              if (c < count) cp_async16(to + 4 * S::ARRAY + (c * 32 + lane) * 16, from + c * a.N);
          }
          // The warp's tokens of B and C.
          const int i = warp * 4 + lane / PER, c = lane % PER * V;
#pragma unroll
          for (int q = 0; q < 4 * PER / 32 || q == 0; ++q) {
            const int ii = i + q * (32 / PER);
            const long long u = min(t + ii, a.T_ - 1);
            if (lane < 4 * PER && c % 16 < a.N && (!CARRY || c >= 16))
              cp_async16(vring + stage * S::VECTORS + (ii * 32 + c) * sizeof(T), c < 16 ? pb + u * a.bt + c : pc + u * a.ct + c - 16);
          }
        }
      }
    }
    cp_async_commit();
  };
  const auto land = [&](int stage) {
    if constexpr (SINGLES) {
      unsigned char* to = ring + stage * S::STAGE;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        Raw* at = (Raw*)(to + (4 * r + ln) * S::ROW) + pr;
        at[0] = ex[r];
        at[S::ARRAY / sizeof(Raw)] = ed[r];
        at[2 * S::ARRAY / sizeof(Raw)] = ey[r];
        at[3 * S::ARRAY / sizeof(Raw)] = ez[r];
      }
      if constexpr (ONE) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          ((T*)(vring + stage * S::VECTORS))[(4 * warp + i) * 32 + lane] = lane % 16 < a.N ? ev[i] : narrow<T>(0.f);
        if constexpr (!CARRY) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
            *(float4*)(to + 4 * S::ARRAY + (c * 32 + lane) * 16) = make_float4(ek[c][0].x, ek[c][0].y, ek[c][1].x, ek[c][1].y);
        }
      }
    }
  };
  if constexpr (!SINGLES) {  // states past the last, and channels, stay zero
    for (int k = lane; k < S::STAGES * S::STAGE / 16; k += 32) ((float4*)ring)[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = threadIdx.x; k < S::STAGES * S::VECTORS / 16; k += kSscThreads) ((float4*)vring)[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
  }

  unsigned flag = 0, dropped = 0;
  int stage = 0;
  fetch(tile1 - 1, 0);
  land(0);
  for (int tile = tile1 - 1; tile >= tile0; --tile) {
    const int t0 = tile * L, number = (tile1 - 1 - tile) % 32;
    if (number == 0) flag = flags(tile);
    const unsigned starts = __shfl_sync(0xffffffffu, flag, number);
    dropped |= starts;
    cp_async_wait<0>();
    __syncwarp();
    const unsigned char* raw = ring + stage * S::STAGE;
    // Tokens behind the last are left out, since 0 times a rate, a b or a c may be a NaN.  (No token before
    // them needs their states.)
    const int left = a.T_ - t0;
    const bool whole = t0 + L <= a.T_;
    const auto pair = [&](int array, int t) { return P::wide(((const Raw*)(raw + array * S::ARRAY + t * S::ROW))[pr]); };
    // A
    float size = 0.f;  // not finite where an input is not
    if constexpr (!ONE) {
      for (int k = threadIdx.x; k < NB * L * 32; k += kSscThreads) {
        const int n = k % 16, second = k / 16 % 2, i = k / 32 % L, n0 = k / (32 * L) * 16 + n;
        const long long u = min(t0 + i, a.T_ - 1);
        const float v = n0 < a.N ? widen(second ? pc[u * a.ct + n0] : pb[u * a.bt + n0]) : 0.f;
        vs[k] = v;
        if (!CARRY) size += fabsf(v);
      }
    } else {
      const int c = threadIdx.x * 4;
      const T* from = (const T*)(vring + stage * S::VECTORS) + (warp * 4 * 32 + lane * 4);
      const float4 v = make_float4(widen(from[0]), widen(from[1]), widen(from[2]), widen(from[3]));
      *(float4*)(vs + c) = v;
      if (!CARRY && special) size = (fabsf(v.x) + fabsf(v.y)) + (fabsf(v.z) + fabsf(v.w));
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int t = 4 * r + ln;
      float2 d = ssc_step_size(a, add2(pair(1, t), bias)), e = pair(2, t);
      if (gated) {
        const float2 z = pair(3, t);
        e = mul2(e, mul2(z, sigmoid<float>(z)));
      }
      float2 u = CARRY ? zero : mul2(d, pair(0, t));
      if (!CARRY && special) size += (fabsf(u.x) + fabsf(u.y)) + (fabsf(e.x) + fabsf(e.y));
      if (!whole && t0 + t >= a.T_) d = e = u = zero;
      du[t * 8 + pr] = make_float4(d.x, d.y, u.x, u.y);
      es[t * 8 + pr] = e;
      if constexpr (CARRY) sum_d = add2(sum_d, d);
    }
    bool wild = false;
    if (!CARRY && special) {
      wild = __syncthreads_or(!(size < __int_as_float(0x7f800000)));
    } else {
      __syncthreads();
    }
    // The other stage has been read: its copies go on behind B.
    stage ^= 1;
    fetch(tile - 1, stage);

    float2 acc[3][ONE ? 1 : R];  // more than 16 states: the own tokens' sums over the blocks
    if constexpr (!ONE && !CARRY) {
#pragma unroll
      for (int w = 0; w < 3; ++w)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[w][r] = zero;
    }
    // C, of own token r.
    const auto finish = [&](int r, float2 along, float2 through, float2 y) {
      const int t = 4 * r + ln, n = whole || t0 + t < a.T_ ? count : 0;
      const long long u = t0 + t;
      const float2 x = pair(0, t), e = es[t * 8 + pr];
      const float4 q = du[t * 8 + pr];
      through = mul2(through, make_float2(kLn2, kLn2));
      float2 dd = fma2(x, along, through);
      if (a.softplus) dd = mul2(dd, sigmoid<float>(add2(pair(1, t), bias)));
      P::store(a.dx + b * a.dxb + u * a.dxt + ch, n, fma2(skip, e, mul2(make_float2(q.x, q.y), along)));
      P::store(a.ddt + b * a.ddtb + u * a.ddtt + ch, n, dd);
      if (t < left) {
        dskip_few = fma2(e, x, dskip_few);
        dbias_few = add2(dbias_few, dd);
      }
      if (gated) {
        const float2 z = pair(3, t), s = sigmoid<T>(z);
        const float2 slope = fma2(mul2(z, s), fma2(s, make_float2(-1.f, -1.f), make_float2(1.f, 1.f)), s);
        P::store(a.dz + b * a.dzb + u * a.dzt + ch, n, mul2(mul2(pair(2, t), fma2(skip, x, y)), slope));
      }
    };

    for (int k = 0; k < NB; ++k) {
      if constexpr (!ONE) {
        rates(k);
        get(2 * k, g);
        get(2 * k + 1, da);
      }
      const float* vk = vs + k * L * 32 + ln * M;
      if constexpr (CARRY) {
        const auto tokens = [&](auto kind) {
          constexpr bool STARTS = decltype(kind)::value != kSscPlain;
#pragma unroll
          for (int t = L - 1; t >= 0; --t) {
            if (decltype(kind)::value == kSscAny && t >= left) continue;
            const float4 q = du[t * 8 + pr], cv = *(const float4*)(vk + t * 32 + 16);
            const float2 e = es[t * 8 + pr];
            const float2 c2[2] = {make_float2(cv.x, cv.y), make_float2(cv.z, cv.w)};
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const float dd = c ? q.y : q.x, ee = c ? e.y : e.x;
                g[c][j] = mul2(ssc_decay(rate[c][j], make_float2(dd, dd)), ssc_fma(make_float2(ee, ee), c2[j], g[c][j]));
                if (STARTS && (starts >> t & 1)) g[c][j] = zero;
              }
          }
        };
        if (!whole) tokens(SscKind<kSscAny>());
        else if (starts) tokens(SscKind<kSscStarts>());
        else tokens(SscKind<kSscPlain>());
      } else {
        float2 h[2][2];
        const auto first_state = [&]() {
          if constexpr (ONE) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float4 q = *(const float4*)(raw + 4 * S::ARRAY + (c * 32 + lane) * 16);
              h[c][0] = make_float2(q.x, q.y), h[c][1] = make_float2(q.z, q.w);
            }
          } else {
            ssc_load_any<M>(a.vec, a.kept + ((b * a.tiles + tile) * a.D + ch) * a.N, k * 16 + ln * M, a.N, count, h);
          }
        };
        const auto tokens = [&](auto kind) {
          constexpr bool STARTS = decltype(kind)::value != kSscPlain, ANY = decltype(kind)::value == kSscAny;
          first_state();
#pragma unroll
          for (int t = 0; t < 12; ++t) {
            const float4 q = du[t * 8 + pr], bv = *(const float4*)(vk + t * 32);
            const float2 b2[2] = {make_float2(bv.x, bv.y), make_float2(bv.z, bv.w)};
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const float dd = c ? q.y : q.x, uu = c ? q.w : q.z;
                if (STARTS && (starts >> t & 1)) h[c][j] = zero;
                h[c][j] = ssc_fma(ssc_decay(rate[c][j], make_float2(dd, dd)), h[c][j], mul2(make_float2(uu, uu), b2[j]));
              }
            if (ANY && wild) clear_past(k, h);
            if ((t & 3) == 3) {
#pragma unroll
              for (int c = 0; c < 2; ++c) save[((t >> 2) * 2 + c) * 32 + lane] = make_float4(h[c][0].x, h[c][0].y, h[c][1].x, h[c][1].y);
            }
          }
#pragma unroll 1
          for (int r = R - 1; r >= 0; --r) {
            float2 before[4][2][2], decay[4][2][2];  // of a token: the state that the one before it left, its decay
            float4 q4[4];
            float2 b2[4][2];
            if (r == 0) {
              first_state();
            } else {
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const float4 q = save[((r - 1) * 2 + c) * 32 + lane];
                h[c][0] = make_float2(q.x, q.y), h[c][1] = make_float2(q.z, q.w);
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int t = 4 * r + i;
              q4[i] = du[t * 8 + pr];
              const float4 bv = *(const float4*)(vk + t * 32);
              b2[i][0] = make_float2(bv.x, bv.y), b2[i][1] = make_float2(bv.z, bv.w);
#pragma unroll
              for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const float dd = c ? q4[i].y : q4[i].x, uu = c ? q4[i].w : q4[i].z;
                  before[i][c][j] = h[c][j];
                  if (STARTS && (starts >> t & 1)) h[c][j] = zero;
                  decay[i][c][j] = ssc_decay(rate[c][j], make_float2(dd, dd));
                  h[c][j] = ssc_fma(decay[i][c][j], h[c][j], mul2(make_float2(uu, uu), b2[i][j]));
                }
              if (ANY && wild) clear_past(k, h), clear_past(k, decay[i]);
            }
#pragma unroll
            for (int i = 3; i >= 0; --i) {
              const int t = 4 * r + i;
              if (ANY && t >= left) continue;  // what would be its sums is not used
              const float4 cv = *(const float4*)(vk + t * 32 + 16);
              const float2 c2[2] = {make_float2(cv.x, cv.y), make_float2(cv.z, cv.w)}, e = es[t * 8 + pr];
              const bool start = STARTS && (starts >> t & 1);
              float2 along[2] = {zero, zero}, through[2] = {zero, zero}, y[2] = {zero, zero};
              float2 vb[2], vc[2];  // dB and dC of the four states, over the pair
              if constexpr (ANY) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                  for (int j = 0; j < 2; ++j) g[c][j] = ssc_fma(c ? make_float2(e.y, e.y) : make_float2(e.x, e.x), c2[j], g[c][j]);
                if (wild) clear_past(k, g);
              }
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const float dd = c ? q4[i].y : q4[i].x, uu = c ? q4[i].w : q4[i].z, ee = c ? e.y : e.x;
                const float2 u2 = make_float2(uu, uu), e2 = make_float2(ee, ee), d2 = make_float2(dd, dd);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const float2 now = i == 3 ? h[c][j] : before[i == 3 ? 0 : i + 1][c][j];  // h_t
                  float2& gg = g[c][j];
                  if constexpr (!ANY) gg = ssc_fma(e2, c2[j], gg);
                  vb[j] = c ? ssc_fma(gg, u2, vb[j]) : mul2(gg, u2);
                  vc[j] = c ? ssc_fma(now, e2, vc[j]) : mul2(now, e2);
                  along[c] = ssc_fma(gg, b2[i][j], along[c]);
                  if (gated) y[c] = ssc_fma(now, c2[j], y[c]);
                  if (start) {
                    gg = zero;
                  } else {
                    gg = mul2(decay[i][c][j], gg);
                    const float2 q = mul2(gg, before[i][c][j]);
                    through[c] = ssc_fma(q, rate[c][j], through[c]);
                    da_few[c][j] = ssc_fma(q, d2, da_few[c][j]);
                  }
                }
              }
              float2* part = sums + ssc_sum_half(i, pr, ln >> 1) + (ln & 1);
              part[0] = make_float2(along[0].x + along[0].y, along[1].x + along[1].y);
              part[128] = make_float2(through[0].x + through[0].y, through[1].x + through[1].y);
              if (gated) part[256] = make_float2(y[0].x + y[0].y, y[1].x + y[1].y);
              // Over the 8 pairs of the warp: a lane keeps value 4 bit2 + 2 bit3 + bit4 of its lane number.
              float v[8] = {vb[0].x, vb[0].y, vb[1].x, vb[1].y, vc[0].x, vc[0].y, vc[1].x, vc[1].y};
              ssc_exchange(v, lane, 4);
              float v4[4] = {v[0], v[1], v[2], v[3]};
              ssc_exchange(v4, lane, 8);
              float v2[2] = {v4[0], v4[1]};
              ssc_exchange(v2, lane, 16);
              red[t * 32 + lane] = v2[0];
            }
            __syncwarp();
            float2 own[3];  // of token 4 r + ln, over the states
#pragma unroll
            for (int w = 0; w < 3; ++w) {
              const float4 lo = *(const float4*)(sums + w * 128 + ssc_sum_half(ln, pr, 0));
              const float4 hi = *(const float4*)(sums + w * 128 + ssc_sum_half(ln, pr, 1));
              own[w] = add2(add2(make_float2(lo.x, lo.y), make_float2(lo.z, lo.w)), add2(make_float2(hi.x, hi.y), make_float2(hi.z, hi.w)));
            }
            if constexpr (ONE) {
              finish(r, own[0], own[1], own[2]);
            } else {
#pragma unroll
              for (int w = 0; w < 3; ++w)
#pragma unroll
                for (int q = 0; q < R; ++q)
                  if (q == r) acc[w][q] = add2(acc[w][q], own[w]);
            }
            __syncwarp();
          }
        };
        if (!whole || wild) tokens(SscKind<kSscAny>());
        else if (starts) tokens(SscKind<kSscStarts>());
        else tokens(SscKind<kSscPlain>());
        // Sums over the part's tokens go over four tiles, then over as many as there are: a chain of all
        // of them would be off by more.
        if (!ONE || (tile & 3) == 0 || tile == tile0) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 2; ++j) da[c][j] = add2(da[c][j], da_few[c][j]), da_few[c][j] = zero;
        }
        __syncthreads();
        // The block's sums for B and C: 16 tokens of 32 values, over the four warps.
        const int which = (lane >> 2 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 4 & 1);
        const int n = k * 16 + ln * M + (which & 3);
        float* out = which < 4 ? a.part_b : a.part_c;
        const float* all = (const float*)((const unsigned char*)red - warp * S::warp_bytes(NB, CARRY));
        const int step = S::warp_bytes(NB, CARRY) / 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = warp * 4 + i;
          const float* r = all + t * 32 + lane;
          const float s = (r[0] + r[step]) + (r[2 * step] + r[3 * step]);
          if (n < a.N && t0 + t < a.T_)
            out[(((block * a.B + b) * a.T_ + t0 + t) * a.G + group) * a.N + n] = s;
        }
        if (!ONE && k + 1 < NB) __syncthreads();  // before the sums are written again
      }
      if constexpr (!ONE) {
        put(2 * k, g);
        put(2 * k + 1, da);
      }
    }
    if constexpr (!ONE && !CARRY) {
#pragma unroll
      for (int r = R - 1; r >= 0; --r) finish(r, acc[0][r], acc[1][r], acc[2][r]);
    }
    if (!CARRY && ((tile & 3) == 0 || tile == tile0)) {
      dskip = add2(dskip, dskip_few), dbias = add2(dbias, dbias_few);
      dskip_few = dbias_few = zero;
    }
    if constexpr (CARRY) __syncthreads();  // before B and C are widened again
    land(stage);
  }

  // The sums over the part's tokens: over the lanes of a pair.
  const auto over_lanes = [&](float2 v) {
#pragma unroll
    for (int bit = 1; bit < 4; bit *= 2) v = add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, bit), __shfl_xor_sync(0xffffffffu, v.y, bit)));
    return v;
  };
  if constexpr (CARRY) {
    const long long q = b * (a.parts - 1) + part - 1;
    const float2 sum = over_lanes(sum_d);
    if (ln == 0) {
      if (count > 0) a.sums[q * a.D + ch] = sum.x;
      if (count > 1) a.sums[q * a.D + ch + 1] = sum.y;
    }
    if (threadIdx.x == 0 && block == 0 && group == 0) a.drops[q] = dropped ? 1.f : 0.f;
    for (int k = 0; k < NB; ++k) {
      if constexpr (!ONE) get(2 * k, g);
      ssc_store_any<M>(a.vec, a.ends + (q * a.D + ch) * a.N, k * 16 + ln * M, a.N, count, g);
    }
  } else {
    float* pa = a.part_a + (b * a.parts + part) * a.D * (a.N + 2);
    for (int k = 0; k < NB; ++k) {
      if constexpr (!ONE) {
        get(2 * k, g);
        get(2 * k + 1, da);
      }
      ssc_store_any<M>(false, pa + (long long)ch * a.N, k * 16 + ln * M, a.N, count, da);
      if (a.dh0 && part == 0) ssc_store_any<M>(a.vec, a.dh0 + row * a.N, k * 16 + ln * M, a.N, count, g);
    }
    dskip = over_lanes(dskip), dbias = over_lanes(dbias);
    if (ln < 2) {
      const float2 v = ln ? dbias : dskip;
      float* out = pa + (long long)a.D * a.N + ln * a.D + ch;
      if (count > 0) out[0] = v.x;
      if (count > 1) out[1] = v.y;
    }
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
  long long sx, sdt, sz, sy, sb, sbg, sc, scg, pool, B;
  unsigned row_blocks;  // blocks of a group of rows
  const float *a, *d, *bias;
  float* state;
  const int32_t* slots;
  int D, N, DG, softplus;
  ErrSink err;
};

// Four lanes a channel, four neighbouring states of each 16 a lane (VEC: as one access of 16
// bytes, and B and C as one of four values).  ROWS = 4: four rows, which share the channel's A and
// keep more loads in flight; what is done once a row and channel is done by one lane for each row.
// 64 rows x 4096 channels x 16 states bf16: 14.3 us of the device, 5.3 of bytes; the latency of one pass from the
// slot to the state and back, at the 512 threads an SM that 126 registers leave (0.37 instructions a cycle).
template <class T, bool VEC, int ROWS>
__global__ void __launch_bounds__(128) ssc_step_kernel(const __grid_constant__ SscStepArgs<T> a) {
  static_assert(ROWS == 1 || ROWS == 4, "a row a lane, or one row");
  pdl_entry();
  const int lane = threadIdx.x & 31, ln = lane & 3;
  // A block takes 32 channels of a group of rows.
  const long long b0 = (long long)(blockIdx.x / a.row_blocks) * ROWS;
  const int place = (int)(blockIdx.x % a.row_blocks) * 32 + (threadIdx.x >> 2);
  const bool live = place < a.D;
  const int ch = live ? place : 0, group = a.DG == a.D ? 0 : ch / a.DG;
  const int rows = live ? (int)min((long long)ROWS, a.B - b0) : 0;
  long long slot[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    slot[r] = -1;
    if (r < rows) slot[r] = a.slots ? (long long)a.slots[b0 + r] : b0 + r;
    if (slot[r] >= a.pool) {  // no such state: reported, and the row treated as padding
      if (ch == 0 && ln == 0) raise_err(a.err, ERRBIT_RANGE);
      slot[r] = -1;
    }
  }
  // The lane's own row (ROWS = 1: each lane the same).
  const int own = ROWS == 1 ? 0 : ln;
  const long long b = b0 + own;
  float x = 0.f, step = 0.f, z = 0.f;
  long long own_slot = slot[0];
#pragma unroll
  for (int r = 1; r < ROWS; ++r) own_slot = own == r ? slot[r] : own_slot;
  if (own_slot >= 0) {
    x = widen(a.x[b * a.sx + ch]);
    const float v = widen(a.dt[b * a.sdt + ch]) + (a.bias ? a.bias[ch] : 0.f);
    if (a.z) z = widen(a.z[b * a.sz + ch]);
    step = a.softplus ? softplus2(make_float2(v, v)).x : v;
  }
  const float* pa = a.a + (long long)ch * a.N;
  float y[ROWS], steps[ROWS], inputs[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    y[r] = 0.f;
    steps[r] = ROWS == 1 ? step : __shfl_sync(0xffffffffu, step, (lane & ~3) | r);
    inputs[r] = ROWS == 1 ? step * x : __shfl_sync(0xffffffffu, step * x, (lane & ~3) | r);
  }
  for (int n0 = ln * 4; n0 < a.N; n0 += 16) {
    float w[4], h[ROWS][4];
    T vb[ROWS][4], vc[ROWS][4];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (slot[r] >= 0) {
        const float* ps = a.state + (slot[r] * a.D + ch) * a.N + n0;
        const T *pb = a.b + (b0 + r) * a.sb + group * a.sbg + n0, *pc = a.c + (b0 + r) * a.sc + group * a.scg + n0;
        if constexpr (VEC) {
          const float4 q = *(const float4*)ps;
          h[r][0] = q.x, h[r][1] = q.y, h[r][2] = q.z, h[r][3] = q.w;
          using Four = std::conditional_t<sizeof(T) == 4, float4, uint2>;
          const Four fb = *(const Four*)pb, fc = *(const Four*)pc;
          memcpy(vb[r], &fb, sizeof(fb));
          memcpy(vc[r], &fc, sizeof(fc));
        } else {
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            if (n0 + s < a.N) h[r][s] = ps[s], vb[r][s] = pb[s], vc[r][s] = pc[s];
          }
        }
      }
    }
    if constexpr (VEC) {
      const float4 q = *(const float4*)(pa + n0);
      w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s) w[s] = n0 + s < a.N ? pa[n0 + s] : 0.f;
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) w[s] *= kLog2e;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (slot[r] >= 0) {
        float* ps = a.state + (slot[r] * a.D + ch) * a.N + n0;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          if (VEC || n0 + s < a.N) {
            h[r][s] = fmaf(ex2(fmaf(steps[r], w[s], kSscCentre)), h[r][s], inputs[r] * widen(vb[r][s]));
            y[r] = fmaf(h[r][s], widen(vc[r][s]), y[r]);
          }
        }
        if constexpr (VEC) {
          *(float4*)ps = make_float4(h[r][0], h[r][1], h[r][2], h[r][3]);
        } else {
#pragma unroll
          for (int s = 0; s < 4; ++s)
            if (n0 + s < a.N) ps[s] = h[r][s];
        }
      }
    }
  }
  // Over the four lanes: each ends with its own row's sum.
  float sum;
  if constexpr (ROWS == 1) {
    sum = y[0] + __shfl_xor_sync(0xffffffffu, y[0], 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
  } else {
    float v[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float send = ln & 1 ? y[2 * q] : y[2 * q + 1], keep = ln & 1 ? y[2 * q + 1] : y[2 * q];
      v[q] = keep + __shfl_xor_sync(0xffffffffu, send, 1);
    }
    const float send = ln & 2 ? v[0] : v[1], keep = ln & 2 ? v[1] : v[0];
    sum = keep + __shfl_xor_sync(0xffffffffu, send, 2);
  }
  if (own < rows && (ROWS > 1 || ln == 0)) {
    if (own_slot >= 0) {
      if (a.d) sum = fmaf(a.d[ch], x, sum);
      if (a.z) sum *= z * sigmoid<T>(make_float2(z, z)).x;
    } else {
      sum = 0.f;
    }
    a.y[b * a.sy + ch] = narrow<T>(sum);
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
  for (const void* q : {(const void*)j.a, (const void*)j.h0, (const void*)j.last, (const void*)j.kept, (const void*)j.dlast, (const void*)j.dh0}) a.vec = a.vec && (uintptr_t)q % 16 == 0;
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
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kernel, (unsigned)grid, kSscThreads, smem, ctx.stream, a);
}

template <class T, SscMode MODE, bool ONE, int LN> cudaError_t ssc_forward(const SelectiveScanJob& j, const SscForwardPlan& plan, const LaunchCtx& ctx) {
  const SscArgs<T> a = ssc_args<T>(j, plan.split);
  const long long units = j.B * a.G * ((a.DG + 64 / LN - 1) / (64 / LN));
  const auto grid = [&](long long parts) { return (units * parts + kSscThreads / 32 - 1) / (kSscThreads / 32); };
  using S = SscLane<T, MODE, LN>;
  const int NB = ONE ? 1 : a.NP / 16;
  static_assert(4 * S::warp_bytes(1) == ssc_forward_bytes(sizeof(T), LN, 1) && 4 * S::warp_bytes(8) == ssc_forward_bytes(sizeof(T), LN, 8), "planned with");
  const size_t smem = (size_t)(kSscThreads / 32) * S::warp_bytes(NB);
  profile_before(ctx);
  cudaError_t e = cudaSuccess;
  if (plan.split.parts > 1) e = ssc_launch(ssc_forward_kernel<T, MODE, ONE, true, false, LN>, grid(plan.split.parts - 1), smem, a, ctx);
  if (e == cudaSuccess)
    e = a.N == a.NP ? ssc_launch(ssc_forward_kernel<T, MODE, ONE, false, false, LN>, grid(plan.split.parts), smem, a, ctx)
                    : ssc_launch(ssc_forward_kernel<T, MODE, ONE, false, true, LN>, grid(plan.split.parts), smem, a, ctx);
  profile_after(ctx);
  return e;
}

template <class T, SscMode MODE, bool ONE> cudaError_t ssc_backward(const SelectiveScanJob& j, const LaunchCtx& ctx) {
  const SscSplit split = ssc_backward_split(j.B, j.T, j.D, j.N, j.G, sizeof(T));
  const SscArgs<T> a = ssc_args<T>(j, split);
  const long long units = j.B * a.G * a.blocks;
  profile_before(ctx);
  cudaError_t e = cudaSuccess;
  using S = SscBack<T, MODE>;
  static_assert(S::bytes(1, false) == ssc_backward_bytes(sizeof(T), 1) && S::bytes(8, false) == ssc_backward_bytes(sizeof(T), 8), "planned with");
  if (split.parts > 1)
    e = ssc_launch(ssc_backward_kernel<T, MODE, ONE, true>, units * (split.parts - 1), S::bytes(a.NP / 16, true), a, ctx);
  if (e == cudaSuccess)
    e = ssc_launch(ssc_backward_kernel<T, MODE, ONE, false>, units * split.parts, S::bytes(a.NP / 16, false), a, ctx);
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

template <class T, SscMode MODE> cudaError_t ssc_forward_any(const SelectiveScanJob& j, const LaunchCtx& ctx) {
  const SscForwardPlan plan = ssc_forward_plan(j.B, j.T, j.D, j.N, j.G, sizeof(T), MODE == kSscSingles);
  if (j.N > 16) return ssc_forward<T, MODE, false, 4>(j, plan, ctx);
  return plan.lanes == 2 ? ssc_forward<T, MODE, true, 2>(j, plan, ctx) : ssc_forward<T, MODE, true, 4>(j, plan, ctx);
}
// Whether what is read starts in pieces of V values; written: of a pair.
template <class T> bool ssc_pieces(const SelectiveScanJob& j, int V, std::initializer_list<const SeqArray*> read,
                                   std::initializer_list<const SeqArray*> written) {
  bool even = (j.D / j.G) % V == 0 && j.N % V == 0 && ssc_rows<T>(j.b, V, j.B, j.T, j.G) && ssc_rows<T>(j.c, V, j.B, j.T, j.G);
  for (const SeqArray* s : read) even = even && ssc_rows<T>(*s, V, j.B, j.T);
  for (const SeqArray* s : written) even = even && ssc_rows<T>(*s, 2, j.B, j.T);
  return even;
}
template <class T> cudaError_t launch_selective_scan(const SelectiveScanJob& j, const LaunchCtx& ctx) {
  const auto pieces = [&](int V) { return ssc_pieces<T>(j, V, {&j.x, &j.dt, &j.z}, {&j.y}); };
  if (pieces(16 / sizeof(T))) return ssc_forward_any<T, kSscWhole>(j, ctx);
  if constexpr (sizeof(T) == 2) {
    if (!pieces(2)) return ssc_forward_any<T, kSscSingles>(j, ctx);
  }
  return ssc_forward_any<T, kSscWords>(j, ctx);
}

template <class T, SscMode MODE> cudaError_t ssc_backward_any(const SelectiveScanJob& j, const LaunchCtx& ctx) {
  return j.N <= 16 ? ssc_backward<T, MODE, true>(j, ctx) : ssc_backward<T, MODE, false>(j, ctx);
}
template <class T> cudaError_t launch_selective_scan_backward(const SelectiveScanJob& j, const LaunchCtx& ctx) {
  const auto pieces = [&](int V) { return ssc_pieces<T>(j, V, {&j.x, &j.dt, &j.z, &j.dy}, {&j.dx, &j.ddt, &j.dz}); };
  if (pieces(16 / sizeof(T)) && (uintptr_t)j.kept % 16 == 0) return ssc_backward_any<T, kSscWhole>(j, ctx);
  if constexpr (sizeof(T) == 2) {
    if (!pieces(2)) return ssc_backward_any<T, kSscSingles>(j, ctx);
  }
  return ssc_backward_any<T, kSscWords>(j, ctx);
}

template <class T> cudaError_t launch_selective_scan_step(const SelectiveScanStepJob& j, const LaunchCtx& ctx) {
  SscStepArgs<T> a = {};
  a.x = (const T*)j.x, a.dt = (const T*)j.dt, a.z = (const T*)j.z, a.b = (const T*)j.b, a.c = (const T*)j.c;
  a.y = (T*)j.y;
  a.sx = j.sx, a.sdt = j.sdt, a.sz = j.sz, a.sy = j.sy, a.sb = j.sb, a.sbg = j.sbg, a.sc = j.sc, a.scg = j.scg;
  a.a = j.a, a.d = j.d, a.bias = j.bias, a.state = j.state, a.slots = j.slots, a.pool = j.pool;
  a.D = (int)j.D, a.N = (int)j.N, a.DG = (int)(j.D / j.G), a.softplus = j.softplus;
  a.B = j.B;
  a.err = ctx.err;
  const auto four = [&](const void* p, long long row, long long group) {  // four values at once
    return (uintptr_t)p % (4 * sizeof(T)) == 0 && (j.B <= 1 || row % 4 == 0) && (j.G <= 1 || group % 4 == 0);
  };
  const bool vec = j.N % 4 == 0 && (uintptr_t)j.state % 16 == 0 && (uintptr_t)j.a % 16 == 0 && four(j.b, j.sb, j.sbg) &&
                   four(j.c, j.sc, j.scg);
  // Four rows a thread keep more loads in flight, where there are threads enough all the same.
  const bool many = j.B * j.D >= 256ll * ctx.num_sms;
  a.row_blocks = (unsigned)((j.D + 31) / 32);
  const unsigned grid = (unsigned)((many ? (j.B + 3) / 4 : j.B) * a.row_blocks);
  profile_before(ctx);
  cudaError_t e;
  if (many) e = vec ? launch_pdl(ssc_step_kernel<T, true, 4>, grid, 128, 0, ctx.stream, a)
                    : launch_pdl(ssc_step_kernel<T, false, 4>, grid, 128, 0, ctx.stream, a);
  else e = vec ? launch_pdl(ssc_step_kernel<T, true, 1>, grid, 128, 0, ctx.stream, a)
               : launch_pdl(ssc_step_kernel<T, false, 1>, grid, 128, 0, ctx.stream, a);
  profile_after(ctx);
  return e;
}

}  // namespace gbs
