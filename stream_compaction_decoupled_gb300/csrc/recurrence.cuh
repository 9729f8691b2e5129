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
// (EDGE) a strip is narrower by one copy's worth, so that from the boundary below its first
// channel it still fits the same copies, and each lane picks its channels out at the row's
// offset.  A copy never reads outside the array.
//
// Where B*D/64 CTAs would leave SMs idle, a cluster of C CTAs shares the strip: its CTAs
// take C consecutive tiles at a time and send each other their tiles' maps through
// distributed shared memory: asynchronous stores that complete on the receiver's mbarrier,
// which needs no fence behind the CTA's outstanding writes of h as a cluster barrier does.
// The CTAs of a cluster are scheduled together, so the wait ends; it is bounded all the
// same (GB_ERR_TIMEOUT): a thread whose wait ran out neither waits nor sends again, and no
// CTA leaves while others may still send to it.  No global scratch is needed.
//
// The gradient runs the same scan backwards in time.  With g_t = dL/dh_t (all paths) and
// c_t = a_t g_t,   g_t = dh_t + c_{t+1}   and   c_t = a_t c_{t+1} + a_t dh_t,
// which is again a map per row, of a_t and dh_t alone.  Then
//   dx_t = u_t g_t,   df_t = a_t (1 - a_t) h_{t-1} g_t,   di_t = u_t (1 - u_t) x_t g_t,
//   and without i:    df_t = a_t (1 - a_t) (h_{t-1} - x_t) g_t.
// Where starts[t] is set the state before t is dropped: a_t counts as 0 in the scan and
// h_{t-1} as 0 in df_t.  0 times an infinity or a NaN does not drop it, though.  It makes a
// NaN, and what is not finite then never leaves the state again, in any order of composition:
// the state after the last row tells.  Where that is not finite and there are starts, the
// strip is gone through a second time (EXACT), its maps dropping the state by selection (8 x
// 2048 x 2048 bf16 gated with a NaN in every channel 108 us in place of 50.6, gradient 167 in
// place of 85.8).
//
// Measured (GB300, copy rate 6.8 TB/s): 8 x 2048 x 2048 bf16 with i and starts 50.3 us (5.3
// TB/s), its gradient 86.8 us (6.2 TB/s); 1 x 65536 x 2048 254.7 us (4.2 TB/s); gradient of 3 x
// 1537 x 1001 fp32 without i 28.7 us (3.9 TB/s).  The gradient runs at the memory's rate;
// forward, the latency of a round (wait, compose, exchange, replay) shows, more so in a cluster.
#pragma once

#include <cmath>

#include "lm.cuh"
#include "lm.h"
#include "resident.h"

namespace gbs {

// sigmoid(z) and 1 - sigmoid(z) = sigmoid(-z) of two values, each accurate where it is small.
// A NaN stays a NaN.
//
// fp32: e = e^-|z| to 4 units of 2^-24, 1/(1+e) by the instruction, 2 units, and e/(1+e): within
// 8 units from end to end, and 0 and 1 at the ends.
// (8 x 2048 x 2048 gated 82.6 us, by the instructions alone 82.7; 1 x 16384 x 2048 107.3 and
// 103.5.)
//
// 16-bit gates: e = 2^(-z log2 e) with the product rounded once, 1/(1+e) and e/(1+e), by the
// instructions alone: up to 8 + 1.3 |z| units of 2^-24, where the gate itself was rounded to 8
// or 11 bits, which moves either by |z| 2^-9 or |z| 2^-12.  The exponent stops at 2^125, where
// e/(1+e) is still finite; 1/(1+e) ends there, at 2^-125 in place of 0.
template <class T> __device__ __forceinline__ void sigmoid_both(float2 z, float2& s, float2& c) {
  if constexpr (sizeof(T) == 4) {
    const float2 e = exp_full(make_float2(max_nan(-fabsf(z.x), -104.f), max_nan(-fabsf(z.y), -104.f)));
    const float2 d = add2(e, make_float2(1.f, 1.f)), big = make_float2(rcp(d.x), rcp(d.y)), small = mul2(e, big);
    s = make_float2(z.x < 0.f ? small.x : big.x, z.y < 0.f ? small.y : big.y);
    c = make_float2(z.x < 0.f ? big.x : small.x, z.y < 0.f ? big.y : small.y);
  } else {
    const float2 x = mul2(z, make_float2(-kLog2e, -kLog2e));
    const float2 e = make_float2(ex2(min_nan(x.x, 125.f)), ex2(min_nan(x.y, 125.f)));
    const float2 d = add2(e, make_float2(1.f, 1.f));
    s = make_float2(rcp(d.x), rcp(d.y));
    c = mul2(e, s);
  }
}

// sigmoid(z) alone.  16 bits: e may overflow to infinity, which gives 0.
template <class T> __device__ __forceinline__ float2 sigmoid(float2 z) {
  const float2 one = make_float2(1.f, 1.f);
  if constexpr (sizeof(T) == 4) {
    // e^88 is finite; beyond, the result is below the normal numbers and 0.
    const float2 x = make_float2(max_nan(min_nan(-z.x, 88.f), -104.f), max_nan(min_nan(-z.y, 88.f), -104.f));
    const float2 d = add2(exp_full(x), one);
    return make_float2(rcp(d.x), rcp(d.y));
  } else {
    const float2 x = mul2(z, make_float2(-kLog2e, -kLog2e));
    const float2 d = add2(make_float2(ex2(x.x), ex2(x.y)), one);
    return make_float2(rcp(d.x), rcp(d.y));
  }
}

template <class T> struct RecArgs {
  const T *x, *f, *i, *h, *dh;  // backward reads h and dh
  T *y, *dx, *df, *di;          // forward writes y
  long long xb, xt, fb, ft, ib, it, hb, ht, dhb, dht, yb, yt, dxb, dxt, dfb, dft, dib, dit;
  const float *h0, *dlast;
  const uint8_t* starts;
  float *last, *dh0;
  int T_, D, strips;  // strips of W channels per batch row
  ErrSink err;
  unsigned long long wait_ns;
  long long stalled;  // fault injection: the tile whose map is not sent
};

constexpr int kRecMaxCluster = 8;

// R rows a thread, so that a tile of one array is 8 KB whatever the type.
template <class T, bool EDGE_, int STAGES_> struct RecGeom {
  static constexpr bool EDGE = EDGE_;
  static constexpr int STAGES = STAGES_;
  static constexpr int NT = 256, WARPS = NT / 32;
  static constexpr int V = 16 / sizeof(T);                   // values of a copy
  static constexpr int R = 16 / sizeof(T);
  static constexpr int L = WARPS * R;                        // rows of a tile
  static constexpr int W = EDGE ? 64 - V : 64;               // channels of a strip
  // A lane's two channels are neighbours, or EDGE 32 apart: there they are loaded and
  // stored one by one, and the 32 lanes' are neighbours each time.
  static constexpr int APART = EDGE ? 32 : 1;
  static __device__ __forceinline__ int first(int lane) { return EDGE ? lane : 2 * lane; }
  static __device__ __forceinline__ int count(int left) {    // how many of a lane's channels exist
    const int c = left - first(threadIdx.x & 31);
    return c > APART ? 2 : c > 0 ? 1 : 0;
  }
  static constexpr int CHUNKS = 64 / V;                      // copies of a row
  static constexpr int PITCH = CHUNKS * 16;                  // bytes of a row in shared memory
  static constexpr int ARRAY = L * PITCH;
  // EDGE: all lanes load both their channels, at the row's offset of up to 16 bytes less a
  // value.  The last of the 64 then ends past the row, and in the last row of all past the
  // tiles (none of it belongs to a channel that exists): the allocation is that much longer.
  static constexpr int SLACK = EDGE ? 16 : 0;
  static constexpr int REACH = (EDGE ? 16 - (int)sizeof(T) : 0) + (EDGE ? 31 + APART + 1 : 64) * (int)sizeof(T);
  static_assert(REACH <= PITCH + SLACK, "loads stay in the tiles and their slack");
  static constexpr int ROWS = NT / CHUNKS;                   // rows that the CTA copies at once
  static_assert(L == 2 * ROWS, "each thread copies two rows' chunks of each array");
};

// Two channels' map y -> a y + b.  EXACT: where a is -0, which no product of sigmoids is, the
// map drops y whatever it is.
struct RecMap {
  float2 a, b;
};
__device__ __forceinline__ float2 rec_drop() { return make_float2(-0.f, -0.f); }
__device__ __forceinline__ float2 rec_unless(float2 a, float2 v, float drop) {  // v, or `drop` where a is -0
  return make_float2(__float_as_uint(a.x) == 0x80000000u ? drop : v.x, __float_as_uint(a.y) == 0x80000000u ? drop : v.y);
}
template <bool EXACT> __device__ __forceinline__ float2 rec_apply(RecMap m, float2 s) {
  if constexpr (EXACT) s = rec_unless(m.a, s, 0.f);
  return fma2(m.a, s, m.b);
}
// m, then q.
template <bool EXACT> __device__ __forceinline__ RecMap rec_then(RecMap m, RecMap q) {
  if constexpr (EXACT) m = {rec_unless(q.a, m.a, 1.f), rec_unless(q.a, m.b, 0.f)};
  return {mul2(m.a, q.a), fma2(q.a, m.b, q.b)};
}
__device__ __forceinline__ float4 rec_pack(RecMap m) { return make_float4(m.a.x, m.a.y, m.b.x, m.b.y); }
__device__ __forceinline__ RecMap rec_unpack(float4 q) { return {make_float2(q.x, q.y), make_float2(q.z, q.w)}; }

// What threads exchange, in turn over the rounds.  Two slots would do for the CTAs' maps;
// with four the round loop is faster (8 x 2048 x 2048 bf16 gated, gradient: 84.8 us with
// two, 78.4 with four; 1 x 65536 x 2048: 268 and 253, gradient 405 and 364).
constexpr int kRecSlots = 4;
struct RecShared {
  float4 warp[2][8][32];                      // the map of each warp's rows
  float4 cta[kRecSlots][kRecMaxCluster][32];  // the map of each CTA's tile
  float2 carry[2][32];                        // C = 1: the state before the round's rows
  unsigned long long bar[kRecSlots];          // the cluster's maps have arrived
};

// What a thread copies of one array: a chunk of the row p rows after the strip's first in
// scan order (dir = 1: t = p; dir = -1: t = T - 1 - p), of the row ROWS later, and of the
// rows a round of `rows` later.  EDGE: the chunk is the c-th from the boundary below the
// row's channel d0; ROWS and `rows` times a value's size are multiples of 16, so those rows
// all have the same offset, and everything about the chunk but its address is known here.
template <class T, class G> struct RecCopy {
  static_assert(G::ROWS * sizeof(T) % 16 == 0 && G::L * sizeof(T) % 16 == 0 && G::R * sizeof(T) % 16 == 0, "offsets");
  const char* src;       // the chunk of row (tile, tid / CHUNKS)
  long long half, step;  // bytes from row r to r + ROWS, and to the next round's row
  int bytes;             // of a chunk; 0: none of it is in the strip
  bool low;              // EDGE: it may begin before the array
  __device__ __forceinline__ void init(const T* strip, long long st, int t, int dir, long long rows, int d0, int left,
                                       int D) {
    constexpr int es = (int)sizeof(T);
    src = (const char*)(strip + t * st);
    half = dir * G::ROWS * st * (long long)es;
    step = dir * rows * st * (long long)es;
    int at = (int)(threadIdx.x % G::CHUNKS) * 16;  // bytes from d0
    if constexpr (G::EDGE) at -= (int)((uintptr_t)src & 15);
    src += at;
    // A chunk ends with the row, where it does not hold 16 bytes of it.
    bytes = at >= left * es ? 0 : (d0 * es + at + 16 <= D * es ? 16 : left * es - at);
    low = d0 * es + at < 0;
  }
  // The chunk at `from`, if its row is on.  It may begin before the row, in values of the
  // array that no lane looks at; where it would begin before the array, it is taken value
  // by value.
  __device__ __forceinline__ void chunk(unsigned char* dst, const char* from, bool on, const T* array) const {
    if constexpr (!G::EDGE) {
      if (on) cp_async16(dst, from);
    } else {
      if (!on) return;
      if (low && from < (const char*)array) {
#pragma unroll 1
        for (int k = 0; k < bytes / (int)sizeof(T); ++k)
          if ((const T*)from + k >= array) ((T*)dst)[k] = ((const T*)from)[k];
      } else {
        cp_async_part(dst, from, bytes);
      }
    }
  }
  // Both chunks of this round; on0, on1: whether their rows exist.
  __device__ __forceinline__ void fetch(unsigned char* tile, bool on0, bool on1, const T* array) {
    unsigned char* dst = tile + threadIdx.x * 16;  // row tid / CHUNKS, chunk tid % CHUNKS
    chunk(dst, src, on0 && bytes > 0, array);
    chunk(dst + G::ROWS * G::PITCH, src + half, on1 && bytes > 0, array);
    src += step;
  }
};

// The offset of row t of a strip from a 16-byte boundary.  R rows on it is the same, so the
// warps' r-th rows all have that of the r-th row of all.
template <class T, class G> __device__ __forceinline__ unsigned rec_offset(const T* strip, long long st, int t) {
  return G::EDGE ? ((unsigned)(uintptr_t)strip + (unsigned)t * (unsigned)(st * sizeof(T))) & 15 : 0u;
}

// With four rows a warp the offsets are kept in 16 bits, row r at t + dir r; eight are as
// soon worked out each time (1 x 16384 x 2001 gated, gradient, when this was chosen: fp32 209
// us worked out and 197 kept, bf16 155 and 160).
template <class T, class G> __device__ __forceinline__ unsigned rec_keep(const T* strip, long long st, int t, int dir) {
  unsigned kept = 0;
  if constexpr (G::EDGE && sizeof(T) == 4) {
#pragma unroll
    for (int r = 0; r < G::R; ++r) kept |= rec_offset<T, G>(strip, st, t + dir * r) << 4 * r;
  }
  return kept;
}
template <class T, class G>
__device__ __forceinline__ unsigned rec_offset(unsigned kept, int r, const T* strip, long long st, int t) {
  if constexpr (G::EDGE && sizeof(T) == 4) return kept >> 4 * r & 15;
  else return rec_offset<T, G>(strip, st, t);
}

// A lane's two channels of row `r` of a tile, whose offset is `off`.
template <class T, class G> __device__ __forceinline__ float2 rec_pair(const unsigned char* tile, int r, unsigned off) {
  const int lane = threadIdx.x & 31;
  const unsigned char* row = tile + r * G::PITCH;
  if constexpr (!G::EDGE) {
    if constexpr (sizeof(T) == 4) {
      return *(const float2*)(row + lane * 8);
    } else {
      return widen2<T>(*(const unsigned*)(row + lane * 4));
    }
  } else {
    const T* q = (const T*)(row + off) + G::first(lane);
    return make_float2(widen(q[0]), widen(q[G::APART]));
  }
}

// Writes a lane's two channels of a row, the first at p; n of them (0 .. 2) exist.
template <class T, class G> __device__ __forceinline__ void rec_store(T* p, float2 v, int n) {
  if constexpr (!G::EDGE) {
    if (n > 0) {
      if constexpr (sizeof(T) == 4) {
        *(float2*)p = v;
      } else {
        *(unsigned*)p = narrow2<T>(v);
      }
    }
  } else {
    if (n > 0) p[0] = narrow<T>(v.x);
    if (n > 1) p[G::APART] = narrow<T>(v.y);
  }
}
template <class G> __device__ __forceinline__ float2 rec_load2(const float* p, int n) {
  return make_float2(n > 0 ? p[0] : 0.f, n > 1 ? p[G::APART] : 0.f);
}
template <class G> __device__ __forceinline__ void rec_store2(float* p, float2 v, int n) {
  if (n > 0) p[0] = v.x;
  if (n > 1) p[G::APART] = v.y;
}

// Makes the cluster's mbarriers and waits until every CTA of it has.
__device__ __forceinline__ void rec_cluster_init(RecShared& sh, unsigned C) {
  if (C == 1) return;
  if (threadIdx.x == 0) {
    for (int k = 0; k < kRecSlots; ++k) mbar_init(&sh.bar[k], 1);
    fence_mbar_init();
  }
  cluster_sync();
}

// Before a CTA of a cluster leaves.  No CTA sends after the barrier, and one whose waits
// all ended has had everything that was sent to it.  Where a wait ran out (`late`, of this
// thread) stores may be on their way still: they land within a microsecond or two, and the
// CTA stays for twenty.
__device__ __forceinline__ void rec_cluster_leave(unsigned C, bool late) {
  if (C == 1) return;
  cluster_sync_relaxed();
  if (late) {
    cp_async_wait<0>();
    const unsigned long long t0 = globaltimer();
    while (globaltimer() - t0 < 20000) __nanosleep(1000);
  }
}

// The states (two channels) that this warp's first row starts from, given the map m of its
// rows.  `carry` is the state before the cluster's rows of this round, moved past them in
// warp 7 (C = 1, where the others read it from shared memory) or in all (C > 1).  `late` is
// set where the wait for the cluster's maps ran out; the rounds left are then gone through
// without, with whatever the slots hold.  (Leaving the loop instead, by a shared flag read
// each round, took 10% more time: 8 x 2048 x 2048 bf16 gated 54.8 us against 50.2, its
// gradient 98.5 against 86.2.)  All threads of the CTA call it.
template <bool EXACT, class A>
__device__ __forceinline__ float2 rec_exchange(RecMap m, float2& carry, RecShared& sh, unsigned C, unsigned rank,
                                               int round, bool& late, const A& a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, turn = round & 1, slot = round % kRecSlots;
  if (warp < 7) sh.warp[turn][warp][lane] = rec_pack(m);
  if (C == 1) {
    if (warp == 7) sh.carry[turn][lane] = carry;
    __syncthreads();
    float2 s = sh.carry[turn][lane];
#pragma unroll
    for (int w = 0; w < 7; ++w)
      if (w < warp) s = rec_apply<EXACT>(rec_unpack(sh.warp[turn][w][lane]), s);
    if (warp == 7) carry = rec_apply<EXACT>(m, s);
    return s;
  }
  __syncthreads();
  RecMap before = {make_float2(1.f, 1.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int w = 0; w < 7; ++w)
    if (w < warp) before = rec_then<EXACT>(before, rec_unpack(sh.warp[turn][w][lane]));
  if (warp == 7 && !late) {
    // The CTA's map goes to every CTA of the cluster.  A slot is written again four rounds
    // later: after the sender has had this CTA's map of a later round, which was sent past
    // a barrier that every reader of the slot reached after reading it.
    if (lane == 0) mbar_arrive_expect_tx(&sh.bar[slot], C * 32 * (unsigned)sizeof(float4));
    const float4 all = rec_pack(rec_then<EXACT>(before, m));
    if ((long long)round * C + rank != a.stalled)
      for (unsigned r = 0; r < C; ++r)
        st_async_f4(cluster_addr(&sh.cta[slot][rank][lane], r), all, cluster_addr(&sh.bar[slot], r));
  }
  if (!late && !mbar_wait_cluster(&sh.bar[slot], (unsigned)(round / kRecSlots) & 1, a.wait_ns)) {
    raise_err(a.err, ERRBIT_TIMEOUT);
    late = true;
  }
  float2 s = carry, start = carry;
#pragma unroll
  for (unsigned r = 0; r < kRecMaxCluster; ++r) {
    if (r < C) {
      if (r == rank) start = s;
      s = rec_apply<EXACT>(rec_unpack(sh.cta[slot][r][lane]), s);
    }
  }
  carry = s;
  return rec_apply<EXACT>(before, start);
}

// Whether the strip has to be gone through again: starts, and a state after the last row that
// is not finite in a channel that exists (n of the lane's).  The same for the whole cluster:
// with C > 1 every warp has the state of all 64 channels, else warp 7 does.  All threads of the
// CTA call it; what the round before left in shared memory is free after it.
__device__ __forceinline__ bool rec_again(const uint8_t* starts, float2 carry, int n, unsigned C) {
  if (!starts) return false;
  const bool odd = (n > 0 && !(fabsf(carry.x) < INFINITY)) || (n > 1 && !(fabsf(carry.y) < INFINITY));
  return __syncthreads_or(odd && (C > 1 || threadIdx.x >= 7 * 32));
}

// The same number, which the compiler takes for another one: what the second pass derives from
// it is worked out there, not kept in registers through the first (spills otherwise).
__device__ __forceinline__ unsigned rec_afresh(unsigned v) {
  asm volatile("" : "+r"(v));
  return v;
}

// One pass over the strip: the state after its last row (warp 7, or with C > 1 every warp).
// Rounds count on from round0, as the exchange's slots do.
template <class T, bool GATE, class G, bool EXACT>
__device__ __forceinline__ float2 rec_forward_pass(const RecArgs<T>& a, unsigned C, unsigned char* tiles, RecShared& sh,
                                                   int round0, bool& late) {
  constexpr int R = G::R, NA = GATE ? 3 : 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned rank = C > 1 ? cluster_rank() : 0;
  const unsigned strip = blockIdx.x / C;
  const long long b = strip / a.strips;
  const int d0 = (int)(strip % a.strips) * G::W;
  const int left = a.D - d0 < G::W ? a.D - d0 : G::W;              // channels of this strip
  const int n = G::count(left);                                    // of this lane
  const int step = (int)C * G::L, tile0 = (int)rank * G::L;
  const int rounds = (int)(((long long)a.T_ + step - 1) / step);
  const int mine = tile0 + (int)threadIdx.x / G::CHUNKS;           // the first row this thread copies
  const T *xp = a.x + b * a.xb + d0, *fp = a.f + b * a.fb + d0, *gp = GATE ? a.i + b * a.ib + d0 : nullptr;
  RecCopy<T, G> x, f, g;
  x.init(xp, a.xt, mine, 1, step, d0, left, a.D);
  f.init(fp, a.ft, mine, 1, step, d0, left, a.D);
  if constexpr (GATE) g.init(gp, a.it, mine, 1, step, d0, left, a.D);
  const unsigned xo = rec_keep<T, G>(xp, a.xt, 0, 1), fo = rec_keep<T, G>(fp, a.ft, 0, 1),
                 go = GATE ? rec_keep<T, G>(gp, a.it, 0, 1) : 0;
  T* y = a.y + b * a.yb + d0 + G::first(lane) + (long long)(tile0 + warp * R) * a.yt;
  const long long y_step = step * a.yt;
  const uint8_t* starts = a.starts ? a.starts + b * a.T_ : nullptr;

  auto fetch = [&](int k) {  // this CTA's tile of round k; one commit group a round
    if (k < rounds) {
      unsigned char* base = tiles + (k % G::STAGES) * (NA * G::ARRAY);
      const long long p = (long long)k * step + mine;
      const bool on0 = p < a.T_, on1 = p + G::ROWS < a.T_;
      x.fetch(base, on0, on1, a.x);
      f.fetch(base + G::ARRAY, on0, on1, a.f);
      if constexpr (GATE) g.fetch(base + 2 * G::ARRAY, on0, on1, a.i);
    }
    cp_async_commit();
  };
  // Which of this warp's rows are starts, for 32 rounds at once: lane l has round k + l's,
  // a bit a row.  (A load every round would be waited for together with the copies in
  // flight.)
  auto flags = [&](int k) {
    unsigned bits = 0;
    const long long t = (long long)(k + lane) * step + tile0 + warp * R;
    if (starts) {
#pragma unroll
      for (int r = 0; r < R; ++r) bits |= (t + r < a.T_ && starts[t + r] != 0 ? 1u : 0u) << r;
    }
    return bits;
  };
#pragma unroll
  for (int k = 0; k < G::STAGES - 1; ++k) fetch(k);
  unsigned marks = 0;
  float2 carry = a.h0 ? rec_load2<G>(a.h0 + b * a.D + d0 + G::first(lane), n) : make_float2(0.f, 0.f);
  if constexpr (!EXACT) rec_cluster_init(sh, C);

  for (int k = 0; k < rounds; ++k) {
    const int rows = (int)(a.T_ - (long long)k * step) - tile0 - warp * R;  // rows from this warp's first to the end
    cp_async_wait<G::STAGES - 2>();
    __syncthreads();  // the tile is in; the one before it has been read by all
    fetch(k + G::STAGES - 1);
    if (k % 32 == 0) marks = flags(k);
    const unsigned drop = __shfl_sync(0xffffffffu, marks, k % 32);
    const unsigned char* base = tiles + (k % G::STAGES) * (NA * G::ARRAY) + warp * R * G::PITCH;
    float2 av[R], bv[R];
    auto row = [&](int r) {
      const float2 xs = rec_pair<T, G>(base, r, rec_offset<T, G>(xo, r, xp, a.xt, r));
      const float2 fs = rec_pair<T, G>(base + G::ARRAY, r, rec_offset<T, G>(fo, r, fp, a.ft, r));
      if constexpr (GATE) {
        av[r] = sigmoid<T>(fs);
        bv[r] = mul2(sigmoid<T>(rec_pair<T, G>(base + 2 * G::ARRAY, r, rec_offset<T, G>(go, r, gp, a.it, r))), xs);
      } else {
        float2 u;
        sigmoid_both<T>(fs, av[r], u);
        bv[r] = mul2(u, xs);
      }
    };
    if (rows >= R) {
#pragma unroll
      for (int r = 0; r < R; ++r) row(r);
    } else {
      // Past the end the map is the identity, so that `carry` ends as the last state.
#pragma unroll
      for (int r = 0; r < R; ++r) {
        av[r] = make_float2(1.f, 1.f);
        bv[r] = make_float2(0.f, 0.f);
        if (r < rows) row(r);
      }
    }
    if (drop) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (drop >> r & 1) av[r] = EXACT ? rec_drop() : make_float2(0.f, 0.f);
    }
    RecMap m = {av[0], bv[0]};
#pragma unroll
    for (int r = 1; r < R; ++r) m = rec_then<EXACT>(m, {av[r], bv[r]});
    float2 s = rec_exchange<EXACT>(m, carry, sh, C, rank, round0 + k, late, a);
    T* out = y;
    y += y_step;
    auto write = [&](int r) {
      s = rec_apply<EXACT>({av[r], bv[r]}, s);
      rec_store<T, G>(out, s, n);
      out += a.yt;
    };
    if (rows >= R) {
#pragma unroll
      for (int r = 0; r < R; ++r) write(r);
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r < rows) write(r);
    }
  }
  return carry;
}

// Where in the array this thread's channels are, for the kernels: those that exist, and the
// offset of the first in a (batch, channel) array.
template <class T, class G> __device__ __forceinline__ int rec_where(const RecArgs<T>& a, unsigned C, long long& at) {
  const unsigned strip = blockIdx.x / C;
  const int d0 = (int)(strip % a.strips) * G::W;
  at = (long long)(strip / a.strips) * a.D + d0 + G::first(threadIdx.x & 31);
  return G::count(a.D - d0 < G::W ? a.D - d0 : G::W);
}
template <class T, class G> __device__ __forceinline__ int rec_rounds(const RecArgs<T>& a, unsigned C) {
  return (int)(((long long)a.T_ + (int)C * G::L - 1) / ((int)C * G::L));
}

template <class T, bool GATE, class G>
__global__ void __launch_bounds__(G::NT, 2) rec_forward_kernel(const __grid_constant__ RecArgs<T> a, unsigned C) {
  extern __shared__ __align__(16) unsigned char tiles[];
  __shared__ RecShared sh;
  pdl_entry();
  bool late = false;
  float2 carry = rec_forward_pass<T, GATE, G, false>(a, C, tiles, sh, 0, late);
  long long at;
  const int n = rec_where<T, G>(a, C, at);
  if (rec_again(a.starts, carry, n, C)) {
    const unsigned C2 = rec_afresh(C);
    carry = rec_forward_pass<T, GATE, G, true>(a, C2, tiles, sh, rec_rounds<T, G>(a, C2), late);
  }
  if (a.last && blockIdx.x % C == 0 && threadIdx.x >= 7 * 32) rec_store2<G>(a.last + at, carry, n);
  rec_cluster_leave(C, late);
}

// Position p = 0, 1, ... counts rows from the end: t = T - 1 - p.
template <class T, bool GATE, class G, bool EXACT>
__device__ __forceinline__ float2 rec_backward_pass(const RecArgs<T>& a, unsigned C, unsigned char* tiles, RecShared& sh,
                                                    int round0, bool& late) {
  constexpr int R = G::R, NA = GATE ? 5 : 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned rank = C > 1 ? cluster_rank() : 0;
  const unsigned strip = blockIdx.x / C;
  const long long b = strip / a.strips;
  const int d0 = (int)(strip % a.strips) * G::W;
  const int left = a.D - d0 < G::W ? a.D - d0 : G::W;
  const int n = G::count(left);
  const int step = (int)C * G::L, tile0 = (int)rank * G::L;
  const int rounds = (int)(((long long)a.T_ + step - 1) / step);
  const int mine = tile0 + (int)threadIdx.x / G::CHUNKS;
  const T *fp = a.f + b * a.fb + d0, *dhp = a.dh + b * a.dhb + d0, *xp = a.x + b * a.xb + d0,
          *hp = a.h + b * a.hb + d0, *gp = GATE ? a.i + b * a.ib + d0 : nullptr;
  RecCopy<T, G> f, dh, x, h, g;
  const int t_mine = a.T_ - 1 - mine;
  f.init(fp, a.ft, t_mine, -1, step, d0, left, a.D);
  dh.init(dhp, a.dht, t_mine, -1, step, d0, left, a.D);
  x.init(xp, a.xt, t_mine, -1, step, d0, left, a.D);
  h.init(hp, a.ht, t_mine - 1, -1, step, d0, left, a.D);  // h_{t-1}
  if constexpr (GATE) g.init(gp, a.it, t_mine, -1, step, d0, left, a.D);
  const unsigned fo = rec_keep<T, G>(fp, a.ft, a.T_ - 1, -1), dho = rec_keep<T, G>(dhp, a.dht, a.T_ - 1, -1),
                 xo = rec_keep<T, G>(xp, a.xt, a.T_ - 1, -1), ho = rec_keep<T, G>(hp, a.ht, a.T_ - 2, -1),
                 go = GATE ? rec_keep<T, G>(gp, a.it, a.T_ - 1, -1) : 0;
  const int t_warp = a.T_ - 1 - tile0 - warp * R;  // this warp's first row of round 0
  const long long at = b * a.D + d0 + G::first(lane);
  T* dx = a.dx + b * a.dxb + d0 + G::first(lane) + (long long)t_warp * a.dxt;
  T* df = a.df + b * a.dfb + d0 + G::first(lane) + (long long)t_warp * a.dft;
  T* di = GATE ? a.di + b * a.dib + d0 + G::first(lane) + (long long)t_warp * a.dit : nullptr;
  const uint8_t* starts = a.starts ? a.starts + b * a.T_ : nullptr;

  auto fetch = [&](int k) {
    if (k < rounds) {
      unsigned char* base = tiles + (k % G::STAGES) * (NA * G::ARRAY);
      const long long p = (long long)k * step + mine;
      const bool on0 = p < a.T_, on1 = p + G::ROWS < a.T_;
      f.fetch(base, on0, on1, a.f);
      dh.fetch(base + G::ARRAY, on0, on1, a.dh);
      x.fetch(base + 2 * G::ARRAY, on0, on1, a.x);
      h.fetch(base + 3 * G::ARRAY, p + 1 < a.T_, p + G::ROWS + 1 < a.T_, a.h);
      if constexpr (GATE) g.fetch(base + 4 * G::ARRAY, on0, on1, a.i);
    }
    cp_async_commit();
  };
  auto flags = [&](int k) {  // as in the forward kernel
    unsigned bits = 0;
    const long long t = (long long)t_warp - (long long)(k + lane) * step;
    if (starts) {
#pragma unroll
      for (int r = 0; r < R; ++r) bits |= (t - r >= 0 && starts[t - r] != 0 ? 1u : 0u) << r;
    }
    return bits;
  };
#pragma unroll
  for (int k = 0; k < G::STAGES - 1; ++k) fetch(k);
  unsigned marks = 0;
  float2 carry = a.dlast ? rec_load2<G>(a.dlast + at, n) : make_float2(0.f, 0.f);
  const float2 first = a.h0 ? rec_load2<G>(a.h0 + at, n) : make_float2(0.f, 0.f);
  if constexpr (!EXACT) rec_cluster_init(sh, C);

  for (int k = 0; k < rounds; ++k) {
    const int rows = (int)(a.T_ - (long long)k * step) - tile0 - warp * R;  // rows r < rows exist; t = rows - 1 - r
    cp_async_wait<G::STAGES - 2>();
    __syncthreads();
    fetch(k + G::STAGES - 1);
    if (k % 32 == 0) marks = flags(k);
    const unsigned drop = __shfl_sync(0xffffffffu, marks, k % 32);
    const unsigned char* base = tiles + (k % G::STAGES) * (NA * G::ARRAY) + warp * R * G::PITCH;
    float2 s[R], s1[R];  // sigmoid(f) and 1 - sigmoid(f)
    constexpr bool KEEP = G::EDGE && !GATE && !EXACT;  // keep dh, whose place takes some working out, where registers allow
    float2 kept[KEEP ? R : 1];
    // Row r's map is c -> a (dh + c).  The sum (dh + c of the rows so far, from c = 0) is kept
    // one row ahead of the product, as one fused operation a row; dropped, c is 0.
    RecMap m = {make_float2(1.f, 1.f), make_float2(0.f, 0.f)};
    float2 sum;
    auto past = [&](int r, float2 v, float2 ds) {  // dh_t + a_{t+1} v, row r - 1 being t + 1
      const bool dropped = drop >> (r - 1) & 1;
      if (EXACT) return dropped ? ds : fma2(s[r - 1], v, ds);
      return fma2(dropped ? make_float2(0.f, 0.f) : s[r - 1], v, ds);
    };
    auto row = [&](int r) {
      const float2 ds = rec_pair<T, G>(base + G::ARRAY, r, rec_offset<T, G>(dho, r, dhp, a.dht, a.T_ - 1 - r));
      if constexpr (KEEP) kept[r] = ds;
      sigmoid_both<T>(rec_pair<T, G>(base, r, rec_offset<T, G>(fo, r, fp, a.ft, a.T_ - 1 - r)), s[r], s1[r]);
      sum = r ? past(r, sum, ds) : ds;
      // Dropped by the last row too, what is not finite stays in the first pass's map, as above.
      const bool dropped = drop >> r & 1;
      const float2 zero = make_float2(0.f, 0.f);
      m = {mul2(m.a, s[r]), EXACT && dropped ? zero : mul2(!EXACT && dropped ? zero : s[r], sum)};
    };
    if (rows >= R) {
#pragma unroll
      for (int r = 0; r < R; ++r) row(r);
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r < rows) row(r);
    }
    if (drop) m.a = EXACT ? rec_drop() : make_float2(0.f, 0.f);
    const float2 c = rec_exchange<EXACT>(m, carry, sh, C, rank, round0 + k, late, a);  // c_{t+1} of the warp's first row
    T *ox = dx, *of = df, *oi = di;
    dx -= step * a.dxt;
    df -= step * a.dft;
    if constexpr (GATE) di -= step * a.dit;
    float2 gt;  // dL/dh_t
    auto write = [&](int r) {
      const int t = rows - 1 - r;
      const float2 ds = KEEP ? kept[KEEP ? r : 0]
                             : rec_pair<T, G>(base + G::ARRAY, r, rec_offset<T, G>(dho, r, dhp, a.dht, a.T_ - 1 - r));
      const float2 xs = rec_pair<T, G>(base + 2 * G::ARRAY, r, rec_offset<T, G>(xo, r, xp, a.xt, a.T_ - 1 - r));
      float2 hs = t > 0 ? rec_pair<T, G>(base + 3 * G::ARRAY, r, rec_offset<T, G>(ho, r, hp, a.ht, a.T_ - 2 - r)) : first;
      if (drop >> r & 1) hs = make_float2(0.f, 0.f);
      if (r == 0) gt = add2(ds, c);
      else gt = past(r, gt, ds);
      const float2 fg = mul2(mul2(s[r], gt), s1[r]);
      if constexpr (GATE) {
        float2 u, u1;
        sigmoid_both<T>(rec_pair<T, G>(base + 4 * G::ARRAY, r, rec_offset<T, G>(go, r, gp, a.it, a.T_ - 1 - r)), u, u1);
        const float2 ug = mul2(u, gt);
        rec_store<T, G>(ox, ug, n);
        rec_store<T, G>(of, mul2(fg, hs), n);
        rec_store<T, G>(oi, mul2(mul2(ug, u1), xs), n);
      } else {
        rec_store<T, G>(ox, mul2(s1[r], gt), n);
        rec_store<T, G>(of, mul2(fg, make_float2(hs.x - xs.x, hs.y - xs.y)), n);
      }
      ox -= a.dxt;
      of -= a.dft;
      if constexpr (GATE) oi -= a.dit;
    };
    if (rows >= R) {
#pragma unroll
      for (int r = 0; r < R; ++r) write(r);
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r < rows) write(r);
    }
  }
  return carry;
}

template <class T, bool GATE, class G>
__global__ void __launch_bounds__(G::NT, 2) rec_backward_kernel(const __grid_constant__ RecArgs<T> a, unsigned C) {
  extern __shared__ __align__(16) unsigned char tiles[];
  __shared__ RecShared sh;
  pdl_entry();
  bool late = false;
  float2 carry = rec_backward_pass<T, GATE, G, false>(a, C, tiles, sh, 0, late);
  long long at;
  const int n = rec_where<T, G>(a, C, at);
  if (rec_again(a.starts, carry, n, C)) {
    const unsigned C2 = rec_afresh(C);
    carry = rec_backward_pass<T, GATE, G, true>(a, C2, tiles, sh, rec_rounds<T, G>(a, C2), late);
  }
  if (a.dh0 && blockIdx.x % C == 0 && threadIdx.x >= 7 * 32) rec_store2<G>(a.dh0 + at, carry, n);
  rec_cluster_leave(C, late);
}

// One token: row b moves the state slots[b] of the pool on by one step, in place.  A
// negative slot is a padded row: its output is zero and no state moves.  Purely a read
// and a write of each value, one 16-byte pack a thread; 64 rows of 2048 bf16 take 3.5 us,
// a launch and two dependent reads (slot, then state).
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
      float2 s, u;
      if constexpr (GATE) s = sigmoid<T>(make_float2(fs[c], is[c])), u.x = s.y;
      else sigmoid_both<T>(make_float2(fs[c], fs[c]), s, u);
      out[c] = fmaf(s.x, out[c], u.x * xs[c]);
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
  a.T_ = (int)j.T, a.D = (int)j.D;
  return a;
}

// CTAs per cluster.  The strips take as many waves as the clusters that are resident at once
// leave; a wave lasts as long as its rounds (and one to fill the pipeline), and a round
// longer the more CTAs exchange their maps.  The estimate's least is taken.  Measured, both
// directions gated, 5 batch rows of 1500: 60 strips (bf16) 14.1 and 19.2 us in fours, 19.7
// and 25.3 in fives, of which not all are resident; 155 strips 36.6 and 56.1 alone, 39.5 and
// 54.5 in pairs, 35.0 and 48.9 in threes; 255 strips 37.6 and 58.5 alone, 46.4 and 67.8 in
// pairs; 320 strips (fp32) 101 and 173 alone, 99.4 and 158 in pairs.
template <class F> unsigned rec_cluster(long long strips, long long tiles, F&& resident) {
  unsigned best = 1;
  double least = 0;
  for (unsigned c = 1; c <= kRecMaxCluster && c <= tiles; ++c) {
    const long long fit = resident(c);
    if (fit < 1) continue;
    const double t = (double)((strips + fit - 1) / fit) * ((tiles + c - 1) / c + 1) * (1 + 0.12 * (c - 1));
    if (least == 0 || t < least) best = c, least = t;
  }
  return best;
}

template <class G, int NA, class T, class K>
cudaError_t rec_launch(K kernel, const RecurrenceJob& j, RecArgs<T> a, const LaunchCtx& ctx) {
  const long long strips = (j.D + G::W - 1) / G::W;
  a.strips = (int)strips;
  a.err = ctx.err;
  a.wait_ns = ctx.wait_ns;
  a.stalled = ctx.stalled_tile;
  constexpr int smem = G::STAGES * NA * G::ARRAY + G::SLACK;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // What is resident is a property of this kernel (each instance launches one) and the device.
  static ResidentTable<kMaxDevices, kRecMaxCluster> resident;
  const unsigned C = rec_cluster(strips * j.B, (j.T + G::L - 1) / G::L, [&](unsigned c) {
    return resident.get(ctx.device, c, [&](unsigned size) {
      return size == 1 ? 2 * ctx.num_sms : clusters_resident(kernel, G::NT, size, smem);
    });
  });
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
