// causal_conv.cuh -- a short causal convolution of each channel over time, its gradient, and
// its form for one token a call on a pool of states.
//
//   p_t = bias + sum_{j < taps} w_{taps-1-j} x_{t-j},   y_t = p_t sigmoid(p_t), or p_t,
//
// x before token 0 from the state (zero without), and x_{t-j} = 0 where a document starts in
// (t - j, t].  The gradient, with q_t = dy_t act'(p_t):
//   dx_t = sum_j w_{taps-1-j} q_{t+j} [no start in (t, t + j]],   dw_{taps-1-j} = sum_t q_t x_{t-j},
//   dbias = sum_t q_t.
//
// Bound by memory: x in and y out (dy and x in, dx out), a few packed operations an element.
// A warp takes 32 V neighbouring channels and a run of tokens; a lane's V channels lie side by
// side where all rows allow vectors of them, or 32 apart, where single values of 32 lanes are
// neighbours.  The window of inputs moves along in registers, so x is read once but for the
// taps - 1 tokens before a run (the gradient: and after it).  How far the window reaches back
// into its document is one number for the whole warp: `age`, the tokens since the start.  What a
// warp reads comes by asynchronous copies into a ring of its own in shared memory (registers alone
// held too few bytes in flight: 8 x 2048 x 2048 bf16 49 us), or, where rows are not on 16-byte
// boundaries, by loads a group of tokens ahead.
//
// Measured (GB300, cold caches): 8 x 2048 x 2048, 4 taps, bf16, with starts 33.9 us (0.58 of the copy rate),
// its gradient 64.6 us (0.46): registers allow 16 and 12 warps an SM, and the chain from the
// products through the gate leaves half the issue slots empty.
#pragma once

#include "lm.cuh"
#include "lm.h"

namespace gbs {

template <class T> struct ConvArgs {
  const T *x, *dy, *state, *dlast;
  T *y, *dx, *last, *dstate;
  const void *w, *bias;
  const uint8_t* starts;
  float* part;
  long long xb, xt, yb, yt, dyb, dyt, dxb, dxt;
  long long units;  // warps' worth of work
  long long B, slots;
  int T_, D, taps, silu, wide;
  int groups, runs, length;
};

__device__ __forceinline__ float conv_param(const void* p, long long k, int wide, float*) {
  return ((const float*)p)[k];
}
template <class T> __device__ __forceinline__ float conv_param(const void* p, long long k, int wide, T*) {
  return wide ? ((const float*)p)[k] : widen(((const T*)p)[k]);
}

// A lane's V values of a row: P side by side, then P of 32 P channels on.  P = V: one access.
// P = 2, 16 bits: words, where rows cannot be read in larger pieces.  P = 1: single values.
template <class T, int V, int P> struct ConvLane {
  static constexpr int GROUPS = V / P;
  using Word = std::conditional_t<P * sizeof(T) == 2, unsigned short,
                                  std::conditional_t<P * sizeof(T) == 4, unsigned, std::conditional_t<P * sizeof(T) == 8, uint2, uint4>>>;
  int first;  // the lane's first channel
  int count;  // how many of the V exist: a multiple of P

  __device__ __forceinline__ ConvLane(int group, int lane, int D) {
    first = group * 32 * V + lane * P;
    const int left = D - first;
    count = left <= 0 ? 0 : P * min(GROUPS, (left + 32 * P - 1) / (32 * P));
  }
  static __device__ __forceinline__ constexpr int place(int e) { return e / P * 32 * P + e % P; }  // from the first
  struct Raw {
    alignas(sizeof(Word)) T v[V];
  };
  __device__ __forceinline__ Raw zero() const {
    Raw r;
#pragma unroll
    for (int e = 0; e < V; ++e) r.v[e] = narrow<T>(0.f);
    return r;
  }
  __device__ __forceinline__ Raw load(const T* row) const {
    Raw r = zero();
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      if (g * P < count) {
        const Word u = *(const Word*)(row + first + g * 32 * P);
        memcpy(r.v + g * P, &u, sizeof(u));
      }
    }
    return r;
  }
  __device__ __forceinline__ void store(T* row, const Raw& r) const {
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      if (g * P < count) {
        Word u;
        memcpy(&u, r.v + g * P, sizeof(u));
        *(Word*)(row + first + g * 32 * P) = u;
      }
    }
  }
  __device__ __forceinline__ void widen_to(const Raw& r, float2 (&f)[V / 2]) const {
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      if constexpr (sizeof(T) == 2) {
        unsigned u;
        memcpy(&u, &r.v[2 * e], 4);
        f[e] = widen2<T>(u);
      } else {
        f[e] = make_float2(r.v[2 * e], r.v[2 * e + 1]);
      }
    }
  }
  __device__ __forceinline__ Raw narrowed(const float2 (&f)[V / 2]) const {
    Raw r;
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      if constexpr (sizeof(T) == 2) {
        const unsigned u = narrow2<T>(f[e]);
        memcpy(&r.v[2 * e], &u, 4);
      } else {
        r.v[2 * e] = f[e].x, r.v[2 * e + 1] = f[e].y;
      }
    }
    return r;
  }
  // Tap or bias values of the lane's channels: p[channel * stride + k].
  __device__ __forceinline__ void params(const void* p, int stride, int k, int wide, float2 (&f)[V / 2]) const {
    float v[V];
#pragma unroll
    for (int e = 0; e < V; ++e)
      v[e] = e < count ? conv_param(p, (long long)(first + place(e)) * stride + k, wide, (T*)nullptr) : 0.f;
#pragma unroll
    for (int e = 0; e < V / 2; ++e) f[e] = make_float2(v[2 * e], v[2 * e + 1]);
  }
};

// The input `back` tokens before token 0 (back >= 1): from the state, or zero.
template <class T, class L>
__device__ __forceinline__ typename L::Raw conv_before(const ConvArgs<T>& a, const L& lane, long long b, int back) {
  const int k = a.taps - 1 - back;
  if (!a.state || k < 0) return lane.zero();
  return lane.load(a.state + (b * (a.taps - 1) + k) * a.D);
}

constexpr int kConvOld = 1 << 20;  // an age past every window

// The window before token t0 (newest last) and how old the document of token t0 - 1 is.
template <class T, int W, class L, int H>
__device__ __forceinline__ int conv_window(const ConvArgs<T>& a, const L& lane, long long b, int t0,
                                           float2 (&hist)[W - 1][H]) {
  int age = kConvOld;
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    const int t = t0 - (W - 1) + k;
    const auto raw = t >= 0 ? lane.load(a.x + b * a.xb + (long long)t * a.xt) : conv_before(a, lane, b, -t);
    lane.widen_to(raw, hist[k]);
    if (a.starts && t >= 0) age = a.starts[b * a.T_ + t] ? 0 : age + 1;
  }
  return age;
}

// Start flags of a run's tokens, 128 at a time (an ordinary load among asynchronous copies waits
// for them): bit k of get(t) is token t + k's, for t that go up by the same divisor of 32 from the
// first.
struct ConvFlags {
  const uint8_t* p;
  int from, end;
  unsigned bits[4] = {0, 0, 0, 0};
  __device__ __forceinline__ ConvFlags(const uint8_t* p_, int t0, int t1) : p(p_), from(t0), end(t1) {
    if (p) read();
  }
  __device__ __forceinline__ void read() {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = from + 32 * k + (int)(threadIdx.x & 31);
      bits[k] = __ballot_sync(0xffffffffu, t < end && p[t] != 0);
    }
  }
  __device__ __forceinline__ unsigned get(int t) {
    if (!p) return 0;
    if (t - from >= 128) {
      from += 128;
      read();
    }
    const int k = (t - from) >> 5;
    const unsigned lo = k & 1 ? bits[1] : bits[0], hi = k & 1 ? bits[3] : bits[2];
    return (k & 2 ? hi : lo) >> ((t - from) & 31);
  }
};

// Where a warp's rows come through: STAGES groups of U rows of each of ARRAYS arrays, copied
// STAGES - 1 groups ahead, in pieces of 16 bytes, or each lane its own words (8 x 2048 x 2046 bf16
// 38.9 us, value by value 41.0; the gradient 67.6 and 86.0).  Single values: one group, in registers
// (fp32 rows are not copied in words: 8 x 2048 x 2047 59.4 us either way, the gradient 94.2 and 98.3).
template <class T, int V, int U, int ARRAYS, int P> struct ConvRing {
  using L = ConvLane<T, V, P>;
  static constexpr bool WHOLE = P == V, SINGLES = P == 1;
  static constexpr int STAGES = 4, ROW = 32 * V * (int)sizeof(T), STAGE = ARRAYS * U * ROW;
  static constexpr int CHUNKS = ROW / 16, ROWS = 32 / CHUNKS;  // 16-byte copies of a row, rows a copy of all lanes
  static constexpr int BYTES = SINGLES ? 0 : STAGES * STAGE;   // a warp
  static_assert(!WHOLE || (ROWS >= 1 && U % ROWS == 0), "whole rows");
  const L& lane;
  unsigned char* ring;
  const T* p[ARRAYS];      // the next group's first row (the lane's part of it)
  long long stride[ARRAYS];
  int next, stop, stage = 0, own_row = 0;
  bool copies = false;
  typename L::Raw raw[SINGLES ? ARRAYS : 1][SINGLES ? U : 1];

  // Rows `first` .. stop - 1; p: row 0 of each array.
  __device__ __forceinline__ ConvRing(const L& lane_, unsigned char* ring_, const T* const (&rows)[ARRAYS],
                                      const long long (&strides)[ARRAYS], int group, int D, int first, int stop_)
      : lane(lane_), ring(ring_), next(first), stop(stop_) {
    const int l = threadIdx.x & 31;
    if constexpr (WHOLE) own_row = l / CHUNKS, copies = group * 32 * V + l % CHUNKS * (16 / (int)sizeof(T)) < D;
#pragma unroll
    for (int k = 0; k < ARRAYS; ++k) {
      stride[k] = strides[k];
      p[k] = rows[k] + (long long)(first + own_row) * strides[k] +
             (WHOLE ? group * 32 * V + l % CHUNKS * (16 / (int)sizeof(T)) : 0);
    }
    if constexpr (SINGLES) {
      fill();
    } else {
#pragma unroll
      for (int s = 0; s < STAGES - 1; ++s) fill();  // groups 0 .. STAGES - 2; the last place is empty
    }
  }
  // Asks for the next group.
  __device__ __forceinline__ void fill() {
    if constexpr (SINGLES) {
#pragma unroll
      for (int k = 0; k < ARRAYS; ++k) {
#pragma unroll
        for (int u = 0; u < U; ++u) raw[k][u] = next + u < stop ? lane.load(p[k] + u * stride[k]) : lane.zero();
        p[k] += U * stride[k];
      }
    } else {
      unsigned char* to = ring + stage * STAGE;
      if constexpr (WHOLE) to += own_row * ROW + (threadIdx.x & 31) % CHUNKS * 16;
      else to += (threadIdx.x & 31) * 4;
#pragma unroll
      for (int k = 0; k < ARRAYS; ++k) {
        if constexpr (WHOLE) {
#pragma unroll
          for (int u = 0; u < U; u += ROWS)
            if (copies && next + u + own_row < stop) cp_async16(to + (k * U + u) * ROW, p[k] + u * stride[k]);
        } else {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const T* row = p[k] + u * stride[k] + lane.first;
#pragma unroll
            for (int g = 0; g < L::GROUPS; ++g)
              if (g * P < lane.count && next + u < stop) cp_async4(to + (k * U + u) * ROW + g * 128, row + g * 32 * P);
          }
        }
        p[k] += U * stride[k];
      }
      cp_async_commit();
      stage = stage == STAGES - 1 ? 0 : stage + 1;
    }
    next += U;
  }
  // The group that was asked for first, widened; asks for another.  Rows from `stop` on are undefined.
  __device__ __forceinline__ void take(float2 (&f)[ARRAYS][U][V / 2]) {
    if constexpr (SINGLES) {
#pragma unroll
      for (int k = 0; k < ARRAYS; ++k)
#pragma unroll
        for (int u = 0; u < U; ++u) lane.widen_to(raw[k][u], f[k][u]);
      fill();  // under way while these are worked on
    } else {
      cp_async_wait<STAGES - 2>();
      __syncwarp();  // the group is there, and the one before it, which is filled again, read by all
      // `stage` is filled next: the group read here is the one after it in the ring.
      const int at = stage == STAGES - 1 ? 0 : stage + 1;
      const unsigned char* from = ring + at * STAGE + (threadIdx.x & 31) * (WHOLE ? V * (int)sizeof(T) : 4);
      fill();
#pragma unroll
      for (int k = 0; k < ARRAYS; ++k)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if constexpr (WHOLE) {
            lane.widen_to(*(const typename L::Raw*)(from + (k * U + u) * ROW), f[k][u]);
          } else {
            typename L::Raw own;
#pragma unroll
            for (int g = 0; g < L::GROUPS; ++g) {
              const unsigned word = *(const unsigned*)(from + (k * U + u) * ROW + g * 128);
              memcpy(own.v + g * P, &word, 4);
            }
            lane.widen_to(own, f[k][u]);
          }
        }
    }
  }
};

template <class T, int W> constexpr int kConvGroup = W == 4 && sizeof(T) == 2 ? 8 : 4;  // tokens of a group

// Blocks of 4 warps an SM, by registers.
template <int W> constexpr int conv_forward_blocks(int P) {
  return P == 1 ? W == 4 ? 3 : 2 : W == 4 && P == 4 ? 4 : 3;
}
template <int W> constexpr int conv_backward_blocks(int P) { return W == 4 && P > 1 ? 3 : 2; }

// Two single operations: beside the gate's exponentials they are quicker than a packed one (forward
// 36.0 -> 33.9 us; the gradient has the same 65 us either way).
__device__ __forceinline__ float2 conv_fma(float2 a, float2 b, float2 c) { return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)); }

template <class T, int W, int V, int P>
__global__ void __launch_bounds__(128, conv_forward_blocks<W>(P)) conv_forward_kernel(const __grid_constant__ ConvArgs<T> a) {
  pdl_entry();
  using L = ConvLane<T, V, P>;
  constexpr int H = V / 2, U = kConvGroup<T, W>;  // tokens whose loads are in flight together
  const long long unit = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (unit >= a.units) return;
  const int group = (int)(unit % a.groups);
  const long long rest = unit / a.groups;
  const int run = (int)(rest % a.runs);
  const long long b = rest / a.runs;
  const L lane(group, threadIdx.x & 31, a.D);
  const int t0 = run * a.length, t1 = min(a.T_, t0 + a.length);
  float2 w[W][H], bias[H], hist[W - 1][H];  // w[j]: the tap of x_{t-j}
#pragma unroll
  for (int j = 0; j < W; ++j) {
    if (j < a.taps) lane.params(a.w, a.taps, a.taps - 1 - j, a.wide, w[j]);
    else
#pragma unroll
      for (int h = 0; h < H; ++h) w[j][h] = make_float2(0.f, 0.f);
  }
#pragma unroll
  for (int h = 0; h < H; ++h) bias[h] = make_float2(0.f, 0.f);
  if (a.bias) lane.params(a.bias, 1, 0, a.wide, bias);
  int age = conv_window<T, W>(a, lane, b, t0, hist);
  T* py = a.y + b * a.yb + (long long)t0 * a.yt;
  ConvFlags flags(a.starts ? a.starts + b * a.T_ : nullptr, t0, t1);
  using Ring = ConvRing<T, V, U, 1, P>;
  extern __shared__ __align__(16) unsigned char conv_shared[];
  Ring ring(lane, conv_shared + (threadIdx.x >> 5) * Ring::BYTES, {a.x + b * a.xb}, {a.xt}, group, a.D, t0, t1);
  for (int t = t0; t < t1; t += U) {
    float2 in[1][U][H], (&xs)[U][H] = in[0];
    ring.take(in);
    const unsigned flag = flags.get(t) & ((1u << U) - 1);
    const auto token = [&](int u, int reach) {
      float2 p[H];
#pragma unroll
      for (int h = 0; h < H; ++h) p[h] = conv_fma(w[0][h], xs[u][h], bias[h]);
#pragma unroll
      for (int j = 1; j < W; ++j) {
        if (j <= reach) {
#pragma unroll
          for (int h = 0; h < H; ++h) p[h] = conv_fma(w[j][h], u >= j ? xs[u >= j ? u - j : 0][h] : hist[u >= j ? 0 : W - 1 + u - j][h], p[h]);
        }
      }
      if (a.silu) {
#pragma unroll
        for (int h = 0; h < H; ++h) p[h] = mul2(p[h], sigmoid<T>(p[h]));
      }
      lane.store(py + u * a.yt, lane.narrowed(p));
    };
    if (flag == 0 && age >= W - 1 && a.taps == W && t + U <= t1) {  // the whole window, four times
#pragma unroll
      for (int u = 0; u < U; ++u) token(u, W - 1);
      age += U;
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t + u < t1) {
          age = flag >> u & 1 ? 0 : age + 1;
          token(u, min(a.taps - 1, age));
        }
      }
    }
    if (t + U <= t1) {
#pragma unroll
      for (int k = 0; k < W - 1; ++k)
#pragma unroll
        for (int h = 0; h < H; ++h) hist[k][h] = k + U < W - 1 ? hist[k + U < W - 1 ? k + U : 0][h] : xs[k + U < W - 1 ? 0 : k + U - (W - 1)][h];
    } else {  // the last tokens of a row: one at a time
      for (int u = 0; u < t1 - t; ++u) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
          for (int h = 0; h < H; ++h) hist[k][h] = k + 1 < W - 1 ? hist[k + 1 < W - 1 ? k + 1 : 0][h] : xs[0][h];
#pragma unroll
        for (int k = 0; k + 1 < U; ++k)
#pragma unroll
          for (int h = 0; h < H; ++h) xs[k][h] = xs[k + 1][h];
      }
    }
    py += U * a.yt;
  }
  if (a.last && t1 == a.T_) {  // the newest inputs, of the last document only
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      const int back = W - 1 - k;  // 1: the newest
      if (back <= a.taps - 1)
        lane.store(a.last + (b * (a.taps - 1) + a.taps - 1 - back) * a.D, back - 1 <= age ? lane.narrowed(hist[k]) : lane.zero());
    }
  }
}

// A run's tokens t0 .. t1 - 1 are its own; it goes W - 1 further for what they take from the
// tokens after them.  pend: dx of the newest W tokens, by their number modulo W.  With very many
// batch rows a warp takes every slots-th of them, so that there are not as many partial sums.
template <class T, int W, int V, int P>
__global__ void __launch_bounds__(128, conv_backward_blocks<W>(P)) conv_backward_kernel(const __grid_constant__ ConvArgs<T> a) {
  pdl_entry();
  using L = ConvLane<T, V, P>;
  constexpr int H = V / 2;
  const long long unit = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (unit >= a.units) return;
  const int group = (int)(unit % a.groups);
  const long long rest = unit / a.groups;
  const int run = (int)(rest % a.runs);
  const L lane(group, threadIdx.x & 31, a.D);
  const int t0 = run * a.length, t1 = min(a.T_, t0 + a.length);
  const float2 zero = make_float2(0.f, 0.f);
  float2 w[W][H], dw[W][H], bias[H], db[H], hist[W - 1][H], pend[W][H];
#pragma unroll
  for (int h = 0; h < H; ++h) bias[h] = db[h] = zero;
#pragma unroll
  for (int j = 0; j < W; ++j) {
#pragma unroll
    for (int h = 0; h < H; ++h) w[j][h] = dw[j][h] = zero;
    if (j < a.taps) lane.params(a.w, a.taps, a.taps - 1 - j, a.wide, w[j]);
  }
  if (a.bias) lane.params(a.bias, 1, 0, a.wide, bias);
  const long long slot = rest / a.runs;
  for (long long b = slot; b < a.B; b += a.slots) {
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int h = 0; h < H; ++h) pend[j][h] = zero;
    int age = conv_window<T, W>(a, lane, b, t0, hist);
    T* po = a.dx + b * a.dxb + (long long)(t0 - (W - 1)) * a.dxt;  // of the token that takes nothing more
    const int end = t1 + W - 1, stop = min(a.T_, end);  // tokens from `stop` on give nothing
    ConvFlags flags(a.starts ? a.starts + b * a.T_ : nullptr, t0, stop);
    using Ring = ConvRing<T, V, W, 2, P>;
    extern __shared__ __align__(16) unsigned char conv_shared[];
    if constexpr (!Ring::SINGLES) {  // the ring's last copies of the row before
      cp_async_wait<0>();
      __syncwarp();
    }
    Ring ring(lane, conv_shared + (threadIdx.x >> 5) * Ring::BYTES, {a.x + b * a.xb, a.dy + b * a.dyb}, {a.xt, a.dyt}, group,
              a.D, t0, stop);
    for (int t = t0; t < end; t += W) {
      float2 in[2][W][H], (&xs)[W][H] = in[0], (&gs)[W][H] = in[1];
      ring.take(in);
      const unsigned flag = flags.get(t) & ((1u << W) - 1);
      const auto token = [&](int u, int reach, bool own) {
        float2 q[H];
        if (a.silu) {
          float2 p[H];
#pragma unroll
          for (int h = 0; h < H; ++h) p[h] = fma2(w[0][h], xs[u][h], bias[h]);
#pragma unroll
          for (int j = 1; j < W; ++j) {
            if (j <= reach) {
#pragma unroll
              for (int h = 0; h < H; ++h) p[h] = fma2(w[j][h], u >= j ? xs[u >= j ? u - j : 0][h] : hist[u >= j ? 0 : W - 1 + u - j][h], p[h]);
            }
          }
#pragma unroll
          for (int h = 0; h < H; ++h) {  // act' = s + p s (1 - s); dw and db may be fp32
            const float2 s = sigmoid<float>(p[h]);
            const float2 c = fma2(s, make_float2(-1.f, -1.f), make_float2(1.f, 1.f));
            q[h] = mul2(gs[u][h], fma2(mul2(p[h], s), c, s));
          }
        } else {
#pragma unroll
          for (int h = 0; h < H; ++h) q[h] = gs[u][h];
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
          if (j <= reach) {
#pragma unroll
            for (int h = 0; h < H; ++h) {
              const float2 xv = u >= j ? xs[u >= j ? u - j : 0][h] : hist[u >= j ? 0 : W - 1 + u - j][h];
              pend[(u - j + W) % W][h] = fma2(w[j][h], q[h], pend[(u - j + W) % W][h]);
              if (own) dw[j][h] = fma2(q[h], xv, dw[j][h]);
            }
          }
        }
        if (own) {
#pragma unroll
          for (int h = 0; h < H; ++h) db[h] = add2(db[h], q[h]);
        }
      };
      // Token t + u - (W - 1) takes nothing more after token t + u.
      const auto inside = [&](int reach) {
#pragma unroll
        for (int u = 0; u < W; ++u) {
          token(u, reach, true);
          float2(&out)[H] = pend[(u + 1) % W];
          lane.store(po + u * a.dxt, lane.narrowed(out));
#pragma unroll
          for (int h = 0; h < H; ++h) out[h] = zero;
        }
        age += W;
      };
      if (flag == 0 && age >= W - 1 && t + W <= t1 && t >= t0 + W - 1) {
        if (a.taps == W) inside(W - 1);
        else inside(a.taps - 1);
      } else {
#pragma unroll
        for (int u = 0; u < W; ++u) {
          if (t + u < stop) {
            age = flag >> u & 1 ? 0 : age + 1;
            token(u, min(a.taps - 1, age), t + u < t1);
          }
          const int done = t + u - (W - 1);
          float2(&out)[H] = pend[(u + 1) % W];
          if (done < t1 && (done >= t0 || (run == 0 && done >= 1 - a.taps))) {
            const int k = done - (a.T_ - (a.taps - 1));  // its place in the last state
            if (a.dlast && k >= 0 && a.T_ - 1 - done <= age) {
              float2 g[H];
              lane.widen_to(lane.load(a.dlast + (b * (a.taps - 1) + k) * a.D), g);
#pragma unroll
              for (int h = 0; h < H; ++h) out[h] = add2(out[h], g[h]);
            }
            if (done >= 0) lane.store(po + u * a.dxt, lane.narrowed(out));
            else if (a.dstate) lane.store(a.dstate + (b * (a.taps - 1) + a.taps - 1 + done) * a.D, lane.narrowed(out));
          }
#pragma unroll
          for (int h = 0; h < H; ++h) out[h] = zero;
        }
      }
#pragma unroll
      for (int k = 0; k < W - 1; ++k)
#pragma unroll
        for (int h = 0; h < H; ++h) hist[k][h] = xs[k + 1][h];
      po += W * a.dxt;
    }
  }
  if (a.part) {  // (run, tap or bias, channel)
    float* p = a.part + (slot * a.runs + run) * (a.taps + 1) * a.D;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
      if (j < a.taps || j == W) {
        float* row = p + (long long)(j == W ? a.taps : a.taps - 1 - j) * a.D;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float2 v = j == W ? db[e / 2] : dw[j == W ? 0 : j][e / 2];
          if (e < lane.count) row[lane.first + L::place(e)] = e % 2 ? v.y : v.x;
        }
      }
    }
  }
}

// Sums the runs' parts, in a fixed order: a block takes 32 values, its 16 warps every 16th run
// and then one warp the 16 sums.
template <class T> struct ConvFoldArgs {
  const float* part;
  void *dw, *db;
  long long rows;  // of parts
  int D, taps, wide;
};
template <class T>
__global__ void __launch_bounds__(512) conv_fold_kernel(const __grid_constant__ ConvFoldArgs<T> a) {
  pdl_entry();
  __shared__ float sums[16][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long width = (long long)(a.taps + 1) * a.D, at = (long long)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (at < width) {
#pragma unroll 8
    for (long long r = warp; r < a.rows; r += 16) s += a.part[r * width + at];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && at < width) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) s += sums[k][lane];
    const int tap = (int)(at / a.D), ch = (int)(at % a.D);
    void* out = tap < a.taps ? a.dw : a.db;
    const long long k = tap < a.taps ? (long long)ch * a.taps + tap : ch;
    if (out) {
      if (a.wide) ((float*)out)[k] = s;
      else ((T*)out)[k] = narrow<T>(s);
    }
  }
}

// ---- one token a call ------------------------------------------------------------------

template <class T> struct ConvStepArgs {
  const T* x;
  T *state, *y;
  const void *w, *bias;
  const int32_t* slots;
  long long sx, sy, pool;
  unsigned row_blocks;  // blocks of a row
  int D, taps, silu, wide, packs;
  bool four;  // 4 taps, which can be read at once
  ErrSink err;
};

// A channel's 4 taps.
template <class T> __device__ __forceinline__ float4 conv_four(const void* p, int ch, int wide) {
  if constexpr (sizeof(T) == 2) {
    if (!wide) {
      const uint2 u = ((const uint2*)p)[ch];
      const float2 lo = widen2<T>(u.x), hi = widen2<T>(u.y);
      return make_float4(lo.x, lo.y, hi.x, hi.y);
    }
  }
  return ((const float4*)p)[ch];
}

// Bound by latency: the slot, then the state and the taps (64 x 4096, 4 taps bf16 9.4 us with cold
// caches, 11.4 with the taps read one by one).
template <class T, int V>
__global__ void __launch_bounds__(128) conv_step_kernel(const __grid_constant__ ConvStepArgs<T> a) {
  pdl_entry();
  const long long b = blockIdx.x / a.row_blocks;
  const int pack = (int)(blockIdx.x % a.row_blocks) * 128 + threadIdx.x;
  if (pack >= a.packs) return;
  const int ch = pack * V;
  long long slot = a.slots ? (long long)a.slots[b] : b;
  if (slot >= a.pool) {  // no such state: reported, and the row treated as padding
    if (ch == 0) raise_err(a.err, ERRBIT_RANGE);
    slot = -1;
  }
  float p[V];
#pragma unroll
  for (int c = 0; c < V; ++c) p[c] = 0.f;
  if (slot >= 0) {
    const Pack<T, V> px = ld_pack<T, V>(a.x + b * a.sx + ch);
    T* st = a.state + slot * (a.taps - 1) * a.D + ch;
    Pack<T, V> old[kConvMaxTaps - 1];
#pragma unroll
    for (int k = 0; k < kConvMaxTaps - 1; ++k)
      if (k < a.taps - 1) old[k] = ld_pack<T, V>(st + (long long)k * a.D);
    if (a.bias) {
#pragma unroll
      for (int c = 0; c < V; ++c) p[c] = conv_param(a.bias, ch + c, a.wide, (T*)nullptr);
    }
    if (a.four) {
      float v[4][V];
#pragma unroll
      for (int k = 0; k < 3; ++k) widen_pack(old[k], v[k]);
      widen_pack(px, v[3]);
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float4 w = conv_four<T>(a.w, ch + c, a.wide);
        p[c] = fmaf(w.w, v[3][c], fmaf(w.z, v[2][c], fmaf(w.y, v[1][c], fmaf(w.x, v[0][c], p[c]))));
      }
    } else {
#pragma unroll
      for (int k = 0; k < kConvMaxTaps; ++k) {
        if (k < a.taps) {
          float v[V];
          if (k == a.taps - 1) widen_pack(px, v);
          else if (k < kConvMaxTaps - 1) widen_pack(old[k < kConvMaxTaps - 1 ? k : 0], v);
#pragma unroll
          for (int c = 0; c < V; ++c)
            p[c] = fmaf(conv_param(a.w, (long long)(ch + c) * a.taps + k, a.wide, (T*)nullptr), v[c], p[c]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kConvMaxTaps - 1; ++k) {
      if (k + 1 < a.taps - 1) st_pack(st + (long long)k * a.D, old[k + 1 < kConvMaxTaps - 1 ? k + 1 : 0]);
      else if (k == a.taps - 2) st_pack(st + (long long)k * a.D, px);
    }
    if (a.silu) {
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float2 s = sigmoid<T>(make_float2(p[c], p[c]));
        p[c] *= s.x;
      }
    }
  }
  st_pack(a.y + b * a.sy + ch, narrow_pack<T, V>(p));
}

// ---- launches --------------------------------------------------------------------------

// Whether vectors of V values can be read and written in every row of the array.
template <class T> bool conv_rows(const SeqArray& s, int V, long long B, long long T_) {
  if (!s.p) return true;
  return (uintptr_t)s.p % (V * sizeof(T)) == 0 && (B <= 1 || s.sb % V == 0) && (T_ <= 1 || s.st % V == 0);
}
template <class T> bool conv_dense(const void* p, int V) { return (uintptr_t)p % (V * sizeof(T)) == 0; }

template <class T> ConvArgs<T> conv_args(const CausalConvJob& j) {
  ConvArgs<T> a = {};
  a.x = (const T*)j.x.p, a.xb = j.x.sb, a.xt = j.x.st;
  a.y = (T*)j.y.p, a.yb = j.y.sb, a.yt = j.y.st;
  a.dy = (const T*)j.dy.p, a.dyb = j.dy.sb, a.dyt = j.dy.st;
  a.dx = (T*)j.dx.p, a.dxb = j.dx.sb, a.dxt = j.dx.st;
  a.w = j.w, a.bias = j.bias, a.wide = j.wide_params;
  a.state = (const T*)j.state, a.last = (T*)j.last, a.dlast = (const T*)j.dlast, a.dstate = (T*)j.dstate;
  a.starts = j.starts;
  a.B = j.B, a.T_ = (int)j.T, a.D = (int)j.D, a.taps = j.taps, a.silu = j.silu;
  return a;
}

template <class K, class T> cudaError_t conv_launch(K kernel, const ConvArgs<T>& a, int smem, const LaunchCtx& ctx) {
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kernel, (unsigned)((a.units + 3) / 4), 128, (size_t)smem, ctx.stream, a);
}

template <class T, int W, int V, int P> cudaError_t conv_forward(const CausalConvJob& j, const LaunchCtx& ctx) {
  ConvArgs<T> a = conv_args<T>(j);
  a.groups = (int)((j.D + 32 * V - 1) / (32 * V));
  // As many warps as fit an SM, and runs of 16 tokens at least: each reads taps - 1 tokens again.
  long long runs = 4ll * conv_forward_blocks<W>(P) * ctx.num_sms / (a.groups * j.B);
  if (runs < 1) runs = 1;
  long long length = (j.T + runs - 1) / runs;
  length = length < 16 ? 16 : (length + 7) / 8 * 8;
  a.length = (int)length;
  a.runs = j.T ? (int)((j.T + length - 1) / length) : 1;
  a.units = j.B * a.runs * a.groups;
  profile_before(ctx);
  const cudaError_t e =
      conv_launch(conv_forward_kernel<T, W, V, P>, a, 4 * ConvRing<T, V, kConvGroup<T, W>, 1, P>::BYTES, ctx);
  profile_after(ctx);
  return e;
}

template <class T, int W, int V, int P> cudaError_t conv_backward(const CausalConvJob& j, const LaunchCtx& ctx) {
  ConvArgs<T> a = conv_args<T>(j);
  a.groups = (int)((j.D + 32 * V - 1) / (32 * V));
  // What fits by registers; with more than 4 taps a warp has 64 channels.
  const ConvSplit s = conv_backward_split(j.B, j.T, j.D, W == 4 ? 4 * conv_backward_blocks<W>(P) : 4);
  a.length = (int)s.length, a.runs = (int)s.runs, a.slots = s.slots;
  a.units = s.slots * a.runs * a.groups;
  a.part = j.dw || j.db ? (float*)j.temp : nullptr;
  profile_before(ctx);
  cudaError_t e =
      conv_launch(conv_backward_kernel<T, W, V, P>, a, 4 * ConvRing<T, V, W, 2, P>::BYTES, ctx);
  if (e == cudaSuccess && a.part) {
    ConvFoldArgs<T> f = {};
    f.part = a.part, f.dw = j.dw, f.db = j.db, f.rows = s.slots * s.runs;
    f.D = a.D, f.taps = j.taps, f.wide = j.wide_params;
    e = launch_pdl(conv_fold_kernel<T>, (unsigned)(((j.taps + 1) * j.D + 31) / 32), 512, 0, ctx.stream, f);
  }
  profile_after(ctx);
  return e;
}

// Rows that are copied in pieces of 16 bytes start on such boundaries, words on theirs.
template <class T> cudaError_t launch_causal_conv(const CausalConvJob& j, const LaunchCtx& ctx) {
  constexpr int V = 4, C = 16 / sizeof(T);
  const auto even = [&](int in, int out) {
    return j.D % in == 0 && conv_rows<T>(j.x, in, j.B, j.T) && conv_rows<T>(j.y, out, j.B, j.T) &&
           conv_dense<T>(j.state, out) && conv_dense<T>(j.last, out);
  };
  if (even(C, V)) return j.taps <= 4 ? conv_forward<T, 4, V, V>(j, ctx) : conv_forward<T, 8, V, V>(j, ctx);
  if constexpr (sizeof(T) == 2) {
    if (even(2, 2)) return j.taps <= 4 ? conv_forward<T, 4, V, 2>(j, ctx) : conv_forward<T, 8, V, 2>(j, ctx);
  }
  return j.taps <= 4 ? conv_forward<T, 4, V, 1>(j, ctx) : conv_forward<T, 8, V, 1>(j, ctx);
}

// (With more than 4 taps a lane has 2 channels.)
template <class T> cudaError_t launch_causal_conv_backward(const CausalConvJob& j, const LaunchCtx& ctx) {
  constexpr int C = 16 / sizeof(T);
  const auto even = [&](int in, int out) {
    return j.D % in == 0 && conv_rows<T>(j.x, in, j.B, j.T) && conv_rows<T>(j.dy, in, j.B, j.T) &&
           conv_rows<T>(j.dx, out, j.B, j.T) && conv_dense<T>(j.state, out) && conv_dense<T>(j.dlast, out) &&
           conv_dense<T>(j.dstate, out);
  };
  if (j.taps > 4) return even(C, 2) ? conv_backward<T, 8, 2, 2>(j, ctx) : conv_backward<T, 8, 2, 1>(j, ctx);
  if (even(C, 4)) return conv_backward<T, 4, 4, 4>(j, ctx);
  if constexpr (sizeof(T) == 2) {
    if (even(2, 2)) return conv_backward<T, 4, 4, 2>(j, ctx);
  }
  return conv_backward<T, 4, 4, 1>(j, ctx);
}

template <class T, int V> cudaError_t conv_step(const CausalConvStepJob& j, const LaunchCtx& ctx) {
  ConvStepArgs<T> a = {};
  a.x = (const T*)j.x, a.sx = j.sx, a.y = (T*)j.y, a.sy = j.sy;
  a.w = j.w, a.bias = j.bias, a.wide = j.wide_params;
  a.state = (T*)j.state, a.pool = j.pool, a.slots = j.slots;
  a.D = (int)j.D, a.taps = j.taps, a.silu = j.silu;
  a.packs = (int)(j.D / V);
  a.row_blocks = (unsigned)((a.packs + 127) / 128);
  a.four = j.taps == 4 && (uintptr_t)j.w % (4 * (j.wide_params ? 4 : sizeof(T))) == 0;
  a.err = ctx.err;
  profile_before(ctx);
  const cudaError_t e = launch_pdl(conv_step_kernel<T, V>, (unsigned)(j.B * a.row_blocks), 128, 0, ctx.stream, a);
  profile_after(ctx);
  return e;
}

template <class T> cudaError_t launch_causal_conv_step(const CausalConvStepJob& j, const LaunchCtx& ctx) {
  constexpr int V = 16 / sizeof(T);
  const bool wide = j.D % V == 0 && conv_dense<T>(j.x, V) && conv_dense<T>(j.y, V) && conv_dense<T>(j.state, V) &&
                    (j.B <= 1 || (j.sx % V == 0 && j.sy % V == 0));
  return wide ? conv_step<T, V>(j, ctx) : conv_step<T, 1>(j, ctx);
}

}  // namespace gbs
