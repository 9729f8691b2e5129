// layer_norm.cuh -- layer norm over the rows of a matrix and its gradient.
//
//   mean = sum x / D,  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps),  n = (x - mean) rstd,
//   y = n w + b;
//   g = dy w:  dx = rstd (g - mean(g) - n mean(g n)),   dw = sum_rows dy n,  db = sum_rows dy.
//
// A row is held in the registers of TPR threads, so it is read once: the mean first, then
// the centred squares (no cancellation), then y.
//
// Rows on 16-byte boundaries (EDGE false) are read and written in whole packs.  Forward,
// such rows take one group of threads each, in no order: the weight comes from L1 and the
// many resident CTAs keep the memory busy.  Otherwise CTAs are persistent: CTA c takes rows
// c + G k (G the grid, a multiple of 8).  Every row of a CTA then starts at the same offset
// from a 16-byte boundary, whatever the width (the offset repeats after at most 8 rows), so
// an odd width is read in whole packs too: they are laid over the row shifted by the
// offset, the first and the last of a row are cut or masked, and the weight, shifted alike,
// is loaded once a CTA.
//
// The gradient's sums over rows stay in the registers of a persistent CTA until it is done;
// one row of partial sums a CTA is then reduced by a second, small launch, in a fixed
// order, so that results do not vary from run to run.
//
// Measured (GB300, copy rate 6.8 TB/s): 16384 x 4096 bf16 45.0 us (6.0 TB/s), gradient 72.0
// us (5.6 TB/s; 8 us of it the second launch); 16773 x 4001 bf16 62.9 and 89.5 us; 16384 x
// 4096 fp32 77.6 and 136.7 us (6.9 and 5.9 TB/s).  Memory bounds it; in 16-bit types the
// issue of some 20 instructions a value comes close.
#pragma once

#include "lm.cuh"
#include "lm.h"

namespace gbs {

template <class T, class P> struct NormArgs {
  const T *x, *dy;
  T *y, *dx;
  long long xs, dys, ys, dxs;  // row strides
  const P *w, *b;
  float *mean, *rstd;          // forward writes them, backward reads them
  float* part;                 // backward: (grid, 2, D) partial sums of dw and db, or null
  long long N;
  int D;
  float eps;
};

// V values a pack, TPR threads a row, NV packs a thread, NT threads a CTA.
template <int V_, int TPR_, int NV_, int NT_, bool EDGE_> struct NormGeom {
  static constexpr int V = V_, TPR = TPR_, NV = NV_, NT = NT_;
  static constexpr bool EDGE = EDGE_;
  static constexpr int ROWS = NT / TPR;       // rows a CTA takes at a time
  static constexpr int WARPS = TPR / 32;      // warps of a row
  static constexpr int STEP = TPR * V;        // values between a thread's packs
};

// Which of a thread's packs lie in a row of D values, all of their values or some.  The
// same for every row of a CTA, so it is worked out once.
template <class G> struct NormPacks {
  unsigned full = 0, part = 0;  // a bit a pack
  int e0, D;                    // the thread's first value
  __device__ __forceinline__ NormPacks(int e0_, int D_) : e0(e0_), D(D_) {
#pragma unroll
    for (int i = 0; i < G::NV; ++i) {
      const int e = e0 + i * G::STEP;
      if (!G::EDGE ? e < D : e >= 0 && e + G::V <= D) full |= 1u << i;
      else if (G::EDGE && e < D && e + G::V > 0) part |= 1u << i;
    }
  }
  __device__ __forceinline__ bool in(int i, int c) const {  // of a part pack
    return (unsigned)(e0 + i * G::STEP + c) < (unsigned)D;
  }
};

// Values e0 .. e0 + V - 1 of a row of D values, the first of them at p; those outside the
// row read as zero.
template <class T, class G> __device__ __forceinline__ Pack<T, G::V> norm_load(const T* p, int e0, int D, bool on) {
  constexpr int V = G::V;
  Pack<T, V> r;
  if constexpr (!G::EDGE) {
    if (on && e0 < D) r = ld_pack<T, V>(p);
    else
#pragma unroll
      for (int c = 0; c < V; ++c) r.v[c] = narrow<T>(0.f);
  } else if (on && e0 >= 0 && e0 + V <= D) {
    r = ld_pack<T, V>(p);
  } else {
#pragma unroll
    for (int c = 0; c < V; ++c) r.v[c] = on && (unsigned)(e0 + c) < (unsigned)D ? p[c] : narrow<T>(0.f);
  }
  return r;
}
// Writes pack i, whose first value goes to p.  A part pack (a thread has two at most, the
// row's first and its last) only goes to `spare`, shared memory of the thread's own, from
// where norm_store_parts writes its values one by one: one copy of that code, after the
// row's registers are free.
template <class T, class G>
__device__ __forceinline__ void norm_store(T* p, const NormPacks<G>& k, int i, const float (&v)[G::V],
                                           unsigned char* spare) {
  if (k.full >> i & 1) st_pack(p, narrow_pack<T, G::V>(v));
  else if (G::EDGE && k.part >> i & 1) st_pack((T*)(spare + (i ? G::NT * 16 : 0)), narrow_pack<T, G::V>(v));
}
template <class T, class G>
__device__ __forceinline__ void norm_store_parts(T* row, const NormPacks<G>& k, const unsigned char* spare) {
  if constexpr (G::EDGE) {
#pragma unroll 1
    for (unsigned left = k.part; left; left &= left - 1) {
      const int i = __ffs(left) - 1;
      const Pack<T, G::V> v = ld_pack<T, G::V>((const T*)(spare + (i ? G::NT * 16 : 0)));
#pragma unroll
      for (int c = 0; c < G::V; ++c)
        if (k.in(i, c)) row[k.e0 + i * G::STEP + c] = v.v[c];
    }
  }
}

// V parameters from e0 on; `none` outside the row and where p is null.
template <class P, class G>
__device__ __forceinline__ void norm_params(P (&r)[G::V], const P* p, int e0, int D, float none) {
  if constexpr (!G::EDGE) {
    if (p && e0 < D) {
      constexpr int N = 16 / sizeof(P);
#pragma unroll
      for (int c = 0; c < G::V; c += N) {
        const uint4 u = *(const uint4*)(p + e0 + c);
        memcpy(r + c, &u, 16);
      }
      return;
    }
#pragma unroll
    for (int c = 0; c < G::V; ++c) r[c] = narrow<P>(none);
  } else {
#pragma unroll
    for (int c = 0; c < G::V; ++c) r[c] = p && (unsigned)(e0 + c) < (unsigned)D ? p[e0 + c] : narrow<P>(none);
  }
}

// Sums of two values over the TPR threads of a row, in a fixed order.  `red` alternates
// between two buffers from call to call, so one barrier a call is enough.
template <class G> struct NormShared {
  float2 red[2][G::ROWS][G::WARPS];
};
template <class G> __device__ __forceinline__ float2 norm_sum(float2 v, NormShared<G>& sh, int& turn) {
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, d);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, d);
  }
  if constexpr (G::WARPS > 1) {
    const int sub = threadIdx.x / G::TPR, w = threadIdx.x % G::TPR / 32;
    if (threadIdx.x % 32 == 0) sh.red[turn][sub][w] = v;
    if constexpr (G::ROWS == 1) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(sub + 1), "n"(G::TPR) : "memory");  // the row's own threads
    v = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < G::WARPS; ++k) {
      const float2 q = sh.red[turn][sub][k];
      v.x += q.x;
      v.y += q.y;
    }
    turn ^= 1;
  }
  return v;
}

// One row's statistics and output from its values in registers (zero outside the row).
template <class T, class P, class G, class W>
__device__ __forceinline__ void norm_row(float (&x)[G::NV][G::V], const NormArgs<T, P>& a, long long row, bool live,
                                         const NormPacks<G>& k, unsigned char* spare, NormShared<G>& sh, int& turn,
                                         W&& params) {
  constexpr int V = G::V, NV = G::NV;
  const float inv = 1.f / (float)a.D;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int c = 0; c < V; ++c) s += x[i][c];
  const float mean = norm_sum<G>(make_float2(s, 0.f), sh, turn).x * inv;
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool full = k.full >> i & 1;
#pragma unroll
    for (int c = 0; c < V; ++c) x[i][c] = full ? x[i][c] - mean : x[i][c];
    if (G::EDGE && k.part >> i & 1) {
#pragma unroll
      for (int c = 0; c < V; ++c) x[i][c] = k.in(i, c) ? x[i][c] - mean : 0.f;
    }
#pragma unroll
    for (int c = 0; c < V; ++c) q = fmaf(x[i][c], x[i][c], q);
  }
  const float rstd = 1.f / sqrtf(norm_sum<G>(make_float2(q, 0.f), sh, turn).x * inv + a.eps);
  if (!live) return;
  if (threadIdx.x % G::TPR == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  T* y = a.y + row * a.ys + k.e0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    P w[V], b[V];
    params(i, w, b);
#pragma unroll
    for (int c = 0; c < V; ++c) x[i][c] = fmaf(x[i][c] * rstd, widen(w[c]), widen(b[c]));
    norm_store<T, G>(y + i * G::STEP, k, i, x[i], spare);
  }
  norm_store_parts<T, G>(a.y + row * a.ys, k, spare);
}

// Rows on 16-byte boundaries.
template <class T, class P, class G>
__global__ void __launch_bounds__(G::NT) norm_forward_kernel(const __grid_constant__ NormArgs<T, P> a) {
  static_assert(!G::EDGE, "whole packs");
  __shared__ NormShared<G> sh;
  pdl_entry();
  const int e0 = (int)(threadIdx.x % G::TPR) * G::V;
  const long long row = (long long)blockIdx.x * G::ROWS + threadIdx.x / G::TPR;
  const bool live = row < a.N;
  const T* p = a.x + row * a.xs + e0;
  Pack<T, G::V> px[G::NV];
#pragma unroll
  for (int i = 0; i < G::NV; ++i) px[i] = norm_load<T, G>(p + i * G::STEP, e0 + i * G::STEP, a.D, live);
  float x[G::NV][G::V];
#pragma unroll
  for (int i = 0; i < G::NV; ++i) widen_pack(px[i], x[i]);
  int turn = 0;
  norm_row<T, P, G>(x, a, row, live, NormPacks<G>(e0, a.D), nullptr, sh, turn, [&](int i, P(&w)[G::V], P(&b)[G::V]) {
    norm_params<P, G>(w, a.w, e0 + i * G::STEP, a.D, 1.f);
    norm_params<P, G>(b, a.b, e0 + i * G::STEP, a.D, 0.f);
  });
}

// A thread's packs of the rows it takes in turn, in shared memory that is its own: filled
// by asynchronous copies STAGES - 1 rows ahead, so that the row in hand costs no registers
// until it is read and the memory stays busy between the reductions.  Packs outside the row
// hold zeros.  No barrier: a thread reads what it copied.
template <class T, class G, int ARRAYS, int STAGES_> struct NormRing {
  static constexpr int STAGES = STAGES_;
  static constexpr int SLOT = G::NT * 16;                       // one pack of every thread
  static constexpr int STAGE = ARRAYS * G::NV * SLOT;
  static constexpr int BYTES = STAGES * STAGE + (G::EDGE ? 2 * SLOT : 0);
  unsigned char* mem;
  __device__ __forceinline__ unsigned char* spare() const { return mem + STAGES * STAGE + threadIdx.x * 16; }
  __device__ __forceinline__ unsigned char* slot(int stage, int array, int i) const {
    return mem + stage * STAGE + (array * G::NV + i) * SLOT + threadIdx.x * 16;
  }
  __device__ __forceinline__ void init(void* smem) {
    mem = (unsigned char*)smem;
    for (int at = threadIdx.x; at < BYTES / 16; at += G::NT) ((uint4*)mem)[at] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
  }
  // The row's pack i: p is where value e0 of the row is, `first` the array's first value.
  // A part pack is copied up to the row's end, zeros after it; what it holds before the
  // row's beginning (values of the array between its rows) is masked when it is read.
  // Only where those would lie before the array are the values taken one by one.
  __device__ __forceinline__ void copy(int stage, int array, int i, const T* p, const T* first,
                                       const NormPacks<G>& k) const {
    if (k.full >> i & 1) {
      cp_async16(slot(stage, array, i), p + i * G::STEP);
    } else if (G::EDGE && k.part >> i & 1) {
      const T* q = p + i * G::STEP;
      T* dst = (T*)slot(stage, array, i);
      const int n = k.D - (k.e0 + i * G::STEP);
      if (q >= first) {
        cp_async_part(dst, q, (n < G::V ? n : G::V) * (int)sizeof(T));
      } else {
#pragma unroll 1
        for (int c = 0; c < G::V; ++c)
          if (k.in(i, c)) dst[c] = q[c];
      }
    }
  }
  __device__ __forceinline__ void read(int stage, int array, int i, float (&v)[G::V], const NormPacks<G>& k) const {
    widen_pack(ld_pack<T, G::V>((const T*)slot(stage, array, i)), v);
    if (G::EDGE && i == 0 && k.e0 < 0) {
#pragma unroll
      for (int c = 0; c < G::V; ++c) v[c] = c < -k.e0 ? 0.f : v[c];
    }
  }
};

// A thread's parameters, laid over the row as its packs are, in shared memory of its own.
template <class P, class G> struct NormParams {
  static constexpr int CHUNKS = G::V * (int)sizeof(P) / 16;
  static constexpr int BYTES = G::NT * G::NV * G::V * (int)sizeof(P);
  unsigned char* mem;
  __device__ __forceinline__ void init(void* smem, const P* p, int e0, int D, float none) {
    mem = (unsigned char*)smem + threadIdx.x * 16;
#pragma unroll
    for (int i = 0; i < G::NV; ++i) {
      P r[G::V];
      norm_params<P, G>(r, p, e0 + i * G::STEP, D, none);
#pragma unroll
      for (int k = 0; k < CHUNKS; ++k) memcpy(mem + (i * CHUNKS + k) * G::NT * 16, (const char*)r + k * 16, 16);
    }
  }
  __device__ __forceinline__ void get(int i, P (&r)[G::V]) const {
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k) {
      const uint4 u = *(const uint4*)(mem + (i * CHUNKS + k) * G::NT * 16);
      memcpy((char*)r + k * 16, &u, 16);
    }
  }
};

// Rows at any offset: persistent, the parameters in shared memory.
template <class T, class P, class G, int STAGES>
__global__ void __launch_bounds__(G::NT) norm_forward_edge_kernel(const __grid_constant__ NormArgs<T, P> a) {
  constexpr int V = G::V, NV = G::NV;
  using Ring = NormRing<T, G, 1, STAGES>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ NormShared<G> sh;
  pdl_entry();
  const long long first = blockIdx.x, grid = gridDim.x;
  if (first >= a.N) return;
  const int t = threadIdx.x % G::TPR, sub = threadIdx.x / G::TPR;
  const int e0 = t * V - (int)((uintptr_t)(a.x + first * a.xs) % 16 / sizeof(T));
  Ring ring;
  ring.init(smem);
  const NormPacks<G> packs(e0, a.D);
  NormParams<P, G> ws, bs;
  ws.init(smem + Ring::BYTES, a.w, e0, a.D, 1.f);
  bs.init(smem + Ring::BYTES + NormParams<P, G>::BYTES, a.b, e0, a.D, 0.f);
  const long long r0 = first + grid * sub, hop = grid * G::ROWS;
  auto fetch = [&](long long row, int stage) {
    if (row < a.N) {
      const T* p = a.x + row * a.xs + e0;
#pragma unroll
      for (int i = 0; i < NV; ++i) ring.copy(stage, 0, i, p, a.x, packs);
    }
    cp_async_commit();
  };
  for (int k = 0; k < STAGES - 1; ++k) fetch(r0 + k * hop, k);
  int turn = 0, stage = 0;
  for (long long row = r0; row < a.N; row += hop) {
    fetch(row + (STAGES - 1) * hop, (stage + STAGES - 1) % STAGES);
    cp_async_wait<STAGES - 1>();
    float x[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) ring.read(stage, 0, i, x[i], packs);
    stage = (stage + 1) % STAGES;
    norm_row<T, P, G>(x, a, row, true, packs, ring.spare(), sh, turn, [&](int i, P(&w)[V], P(&b)[V]) {
      ws.get(i, w);
      bs.get(i, b);
    });
  }
}

// The gradient: persistent, one CTA an SM, x and dy through the ring, the sums over rows in
// registers.  Where those would take too many (32 values a thread, more than 512 threads,
// or 512 at any offset in fp32), db's are in shared memory, each thread's own, and a row's
// n and g are worked out twice; at 32 values the weight comes from L1 in place of shared
// memory.
template <class T, class P, class G> struct NormBackwardSmem {
  static constexpr bool BIG = G::NV * G::V > 16;
  static constexpr bool TIGHT = BIG || G::NT > 512 || (G::EDGE && G::TPR == 512 && G::V == 4);
  static constexpr int SUMS = TIGHT ? G::NT * G::NV * G::V * (int)sizeof(float) : 0;
  static constexpr int ROOM = 220 * 1024, ROW = NormRing<T, G, 2, 1>::STAGE;
  static constexpr int REST = SUMS + (BIG ? 0 : NormParams<P, G>::BYTES) + NormRing<T, G, 2, 1>::BYTES - ROW;
  static constexpr int STAGES = (ROOM - REST) / ROW < 5 ? (ROOM - REST) / ROW : 5;
  using Ring = NormRing<T, G, 2, STAGES>;
  static constexpr int BYTES = STAGES * ROW + REST;
  static_assert(STAGES >= 1, "fits");
};
template <class T, class P, class G>
__global__ void __launch_bounds__(G::NT) norm_backward_kernel(const __grid_constant__ NormArgs<T, P> a) {
  using S = NormBackwardSmem<T, P, G>;
  constexpr int V = G::V, NV = G::NV, N = NV * V, STAGES = S::STAGES;
  constexpr bool BIG = S::BIG, TIGHT = S::TIGHT;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ NormShared<G> sh;
  __shared__ float2 stats[STAGES][G::NT / 32];
  pdl_entry();
  const int t = threadIdx.x % G::TPR, sub = threadIdx.x / G::TPR;
  const long long first = blockIdx.x, grid = gridDim.x;
  const int off = G::EDGE && first < a.N ? (int)((uintptr_t)(a.x + first * a.xs) % 16 / sizeof(T)) : 0;
  const int e0 = t * V - off;
  typename S::Ring ring;
  ring.init(smem);
  const NormPacks<G> packs(e0, a.D);
  float2 dw[N / 2], db_[TIGHT ? 1 : N / 2];
  float2* db_mem = (float2*)(smem + S::Ring::BYTES) + threadIdx.x;
  auto db = [&](int k) -> float2& {
    if constexpr (TIGHT) return db_mem[k * G::NT];
    else return db_[k];
  };
#pragma unroll
  for (int k = 0; k < N / 2; ++k) dw[k] = db(k) = make_float2(0.f, 0.f);
  NormParams<P, G> ws;
  if constexpr (!BIG) ws.init(smem + S::Ring::BYTES + S::SUMS, a.w, e0, a.D, 1.f);
  auto weight = [&](int i, P(&w)[V]) {
    if constexpr (BIG) norm_params<P, G>(w, a.w, e0 + i * G::STEP, a.D, 1.f);
    else ws.get(i, w);
  };
  const float inv = 1.f / (float)a.D;
  const long long r0 = first + grid * sub, hop = grid * G::ROWS;
  auto fetch = [&](long long row, int stage) {
    if (row < a.N) {
      const T *x = a.x + row * a.xs + e0, *dy = a.dy + row * a.dys + e0;
#pragma unroll(G::EDGE ? 1 : NV)
      for (int i = 0; i < NV; ++i) {
        ring.copy(stage, 0, i, x, a.x, packs);
        ring.copy(stage, 1, i, dy, a.dy, packs);
      }
      // The row's statistics come the same way, once a warp: an ordinary load among the
      // copies would be waited for together with all of them (measured: 115.8 us against
      // 88.9 at 16384 x 4096 bf16, with the loads and with constants).
      if (threadIdx.x % 32 == 0) {
        cp_async4(&stats[stage][threadIdx.x / 32].x, a.mean + row);
        cp_async4(&stats[stage][threadIdx.x / 32].y, a.rstd + row);
      }
    }
    cp_async_commit();
  };
  for (int k = 0; k < STAGES - 1; ++k) fetch(r0 + k * hop, k);
  int turn = 0, stage = 0;
  for (long long row = r0; row < a.N; row += hop) {
    fetch(row + (STAGES - 1) * hop, (stage + STAGES - 1) % STAGES);
    cp_async_wait<STAGES - 1>();
    __syncwarp();
    const float mean = stats[stage][threadIdx.x / 32].x, rstd = stats[stage][threadIdx.x / 32].y;
    // n and g = dy w of pack i, two values at a time.
    const float2 m2 = make_float2(-mean, -mean), r2 = make_float2(rstd, rstd);
    auto terms = [&](int i, float2 (&n)[V / 2], float2 (&d)[V / 2], float2 (&g)[V / 2]) {
      float x[V], y[V];
      P w[V];
      ring.read(stage, 0, i, x, packs);
      ring.read(stage, 1, i, y, packs);  // zero outside the row
      weight(i, w);
#pragma unroll
      for (int c = 0; c < V / 2; ++c) {
        n[c] = mul2(add2(make_float2(x[2 * c], x[2 * c + 1]), m2), r2);
        d[c] = make_float2(y[2 * c], y[2 * c + 1]);
        g[c] = mul2(d[c], make_float2(widen(w[2 * c]), widen(w[2 * c + 1])));
      }
    };
    float2 n[TIGHT ? 1 : NV][V / 2], g[TIGHT ? 1 : NV][V / 2];
    float2 sg = make_float2(0.f, 0.f), sgn = sg;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int q = TIGHT ? 0 : i;
      float2 d[V / 2];
      terms(i, n[q], d, g[q]);
#pragma unroll
      for (int c = 0; c < V / 2; ++c) {
        const int k = i * (V / 2) + c;
        dw[k] = fma2(d[c], n[q][c], dw[k]);
        db(k) = add2(db(k), d[c]);
        sg = add2(sg, g[q][c]);
        sgn = fma2(g[q][c], n[q][c], sgn);
      }
    }
    const float2 s = norm_sum<G>(make_float2(sg.x + sg.y, sgn.x + sgn.y), sh, turn);
    const float2 mg = make_float2(-s.x * inv, -s.x * inv), mgn = make_float2(-s.y * inv, -s.y * inv);
    T* dx = a.dx + row * a.dxs + e0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int q = TIGHT ? 0 : i;
      if constexpr (TIGHT) {
        float2 d[V / 2];
        terms(i, n[0], d, g[0]);
      }
      float o[V];
#pragma unroll
      for (int c = 0; c < V / 2; ++c) {
        const float2 v = mul2(add2(fma2(n[q][c], mgn, g[q][c]), mg), r2);
        o[2 * c] = v.x, o[2 * c + 1] = v.y;
      }
      norm_store<T, G>(dx + i * G::STEP, packs, i, o, ring.spare());
    }
    norm_store_parts<T, G>(a.dx + row * a.dxs, packs, ring.spare());
    stage = (stage + 1) % STAGES;
  }
  if (!a.part) return;
  float* part = a.part + (size_t)blockIdx.x * 2 * a.D;
  auto sum = [&](int which, int k) {
    const float2 v = which ? db(k / 2) : dw[k / 2];
    return k % 2 ? v.y : v.x;
  };
  if constexpr (G::ROWS == 1) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int e = e0 + k / V * G::STEP + k % V;
      if ((unsigned)e < (unsigned)a.D) {
        part[e] = sum(0, k);
        part[(size_t)a.D + e] = sum(1, k);
      }
    }
  } else {
    // The CTA's groups of threads, one after another; the ring's memory is free now.
    static_assert(S::Ring::BYTES >= N * G::NT * (int)sizeof(float), "the sums fit");
    float* fold = (float*)smem;
    cp_async_wait<0>();
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < N; ++k) fold[k * G::NT + threadIdx.x] = sum(which, k);
      __syncthreads();
      for (int at = threadIdx.x; at < N * G::TPR; at += G::NT) {
        const int k = at / G::TPR, q = at % G::TPR;
        float v = 0.f;
#pragma unroll
        for (int r = 0; r < G::ROWS; ++r) v += fold[k * G::NT + r * G::TPR + q];
        const int e = q * V - off + k / V * G::STEP + k % V;
        if ((unsigned)e < (unsigned)a.D) part[(size_t)which * a.D + e] = v;
      }
    }
  }
}

// Rows of any alignment and length, value by value: the row is read again for each of
// the passes (from L2).  Rows too long for registers, and arrays whose rows start at
// different offsets from a 16-byte boundary, come here (4096 x 16383 bf16: 103 us, where
// 16384 columns in whole packs take 53).
constexpr int kNormLongThreads = 512;
using NormLongGeom = NormGeom<1, kNormLongThreads, 1, kNormLongThreads, true>;

template <class T, class P>
__global__ void __launch_bounds__(kNormLongThreads) norm_forward_long_kernel(const __grid_constant__ NormArgs<T, P> a) {
  using G = NormLongGeom;
  __shared__ NormShared<G> sh;
  pdl_entry();
  const float inv = 1.f / (float)a.D;
  int turn = 0;
  for (long long row = blockIdx.x; row < a.N; row += gridDim.x) {
    const T* x = a.x + row * a.xs;
    T* y = a.y + row * a.ys;
    float s = 0.f, q = 0.f;
#pragma unroll 8
    for (int e = threadIdx.x; e < a.D; e += G::NT) s += widen(x[e]);
    const float mean = norm_sum<G>(make_float2(s, 0.f), sh, turn).x * inv;
#pragma unroll 8
    for (int e = threadIdx.x; e < a.D; e += G::NT) {
      const float c = widen(x[e]) - mean;
      q = fmaf(c, c, q);
    }
    const float rstd = 1.f / sqrtf(norm_sum<G>(make_float2(q, 0.f), sh, turn).x * inv + a.eps);
    if (threadIdx.x == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
#pragma unroll 4
    for (int e = threadIdx.x; e < a.D; e += G::NT) {
      const float n = (widen(x[e]) - mean) * rstd;
      y[e] = narrow<T>(fmaf(n, a.w ? widen(a.w[e]) : 1.f, a.b ? widen(a.b[e]) : 0.f));
    }
  }
}

template <class T, class P>
__global__ void __launch_bounds__(kNormLongThreads) norm_backward_long_kernel(const __grid_constant__ NormArgs<T, P> a) {
  using G = NormLongGeom;
  __shared__ NormShared<G> sh;
  pdl_entry();
  const float inv = 1.f / (float)a.D;
  int turn = 0;
  for (long long row = blockIdx.x; row < a.N; row += gridDim.x) {
    const T *x = a.x + row * a.xs, *dy = a.dy + row * a.dys;
    T* dx = a.dx + row * a.dxs;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int e = threadIdx.x; e < a.D; e += G::NT) {
      const float g = widen(dy[e]) * (a.w ? widen(a.w[e]) : 1.f);
      s.x += g;
      s.y = fmaf(g, (widen(x[e]) - mean) * rstd, s.y);
    }
    s = norm_sum<G>(s, sh, turn);
    const float mg = s.x * inv, mgn = s.y * inv;
#pragma unroll 4
    for (int e = threadIdx.x; e < a.D; e += G::NT) {
      const float n = (widen(x[e]) - mean) * rstd;
      dx[e] = narrow<T>((fmaf(-n, mgn, widen(dy[e]) * (a.w ? widen(a.w[e]) : 1.f)) - mg) * rstd);
    }
  }
}

// The sums over rows of such arrays: CTA (column block, row range), one column a thread.
template <class T, class P>
__global__ void __launch_bounds__(256) norm_columns_long_kernel(const __grid_constant__ NormArgs<T, P> a, int ranges) {
  pdl_entry();
  const int col = (int)(blockIdx.x / ranges) * 256 + threadIdx.x, range = (int)(blockIdx.x % ranges);
  if (col >= a.D) return;
  float dw = 0.f, db = 0.f;
#pragma unroll 4
  for (long long row = range; row < a.N; row += ranges) {
    const float d = widen(a.dy[row * a.dys + col]);
    dw = fmaf(d, (widen(a.x[row * a.xs + col]) - a.mean[row]) * a.rstd[row], dw);
    db += d;
  }
  float* part = a.part + (size_t)range * 2 * a.D;
  part[col] = dw;
  part[a.D + col] = db;
}

// dw and db from `count` rows of partial sums: 32 columns a CTA, 16 threads a column, whose
// loads are all in flight together.
template <class P>
__global__ void __launch_bounds__(512) norm_fold_kernel(const float* part, int count, int D, P* dw, P* db) {
  __shared__ float red[16][33];
  pdl_entry();
  const int lane = threadIdx.x % 32, g = threadIdx.x / 32;
  const int at = blockIdx.x * 32 + lane;  // a column of (dw, db) side by side
  float s = 0.f;
  if (at < 2 * D) {
#pragma unroll 10
    for (int p = g; p < count; p += 16) s += part[(size_t)p * 2 * D + at];
  }
  red[g][lane] = s;
  __syncthreads();
  if (g == 0 && at < 2 * D) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) s += red[k][lane];
    P* out = at < D ? dw : db;
    if (out) out[at < D ? at : at - D] = narrow<P>(s);
  }
}

// ---- launches ------------------------------------------------------------------------

// Whether rows of the two arrays (null: none) start at equal offsets from a 16-byte
// boundary, for every row.
template <class T> bool same_offsets(const void* p, long long sp, const void* q, long long sq, long long N) {
  return (uintptr_t)p % 16 == (uintptr_t)q % 16 && (N <= 1 || (sp - sq) * (long long)sizeof(T) % 16 == 0);
}

template <class T, class P> NormArgs<T, P> norm_args(const LayerNormJob& j) {
  NormArgs<T, P> a = {};
  a.x = (const T*)j.x, a.xs = j.xs;
  a.y = (T*)j.y, a.ys = j.ys;
  a.dy = (const T*)j.dy, a.dys = j.dys;
  a.dx = (T*)j.dx, a.dxs = j.dxs;
  a.w = (const P*)j.w, a.b = (const P*)j.b;
  a.mean = j.mean, a.rstd = j.rstd;
  a.N = j.N, a.D = (int)j.D, a.eps = j.eps;
  return a;
}

// Whether the rows of an array all start on 16-byte boundaries.
template <class T> bool norm_rows16(const void* p, long long stride, long long N) {
  return (uintptr_t)p % 16 == 0 && (N <= 1 || stride * (long long)sizeof(T) % 16 == 0);
}
inline bool on16(const void* p) { return (uintptr_t)p % 16 == 0; }

// CTAs of a persistent kernel: enough for every row, at most `most`; a multiple of 8.
inline unsigned norm_grid(long long N, long long most) {
  const long long g = N < most ? N : most;
  return (unsigned)((g + 7) / 8 * 8);
}

// Calls f(geometry) with the first of the listed group sizes whose threads hold a row of
// `packs` packs at NV packs a thread; the last one is taken without asking.  A CTA has at
// most MOST threads (or one group), and at most 15 groups that meet at named barriers.
template <int V, int NV, int MOST, bool EDGE, int TPR, int... More, class F>
cudaError_t norm_pick(long long packs, F&& f) {
  if constexpr (sizeof...(More) > 0) {
    if (packs > (long long)TPR * NV) return norm_pick<V, NV, MOST, EDGE, More...>(packs, f);
  }
  constexpr int cap = TPR % 3 == 0 && MOST > 768 ? 768 : MOST;  // whole groups, and 85 registers a thread
  constexpr int fit = cap / TPR < 1 ? 1 : cap / TPR;
  constexpr int rows = TPR > 32 && fit > 15 ? 15 : fit;
  return f((NormGeom<V, TPR, NV, TPR * rows, EDGE>*)nullptr);
}

template <class T, class P> cudaError_t launch_layer_norm(const LayerNormJob& j, const LaunchCtx& ctx) {
  constexpr int V = 16 / sizeof(T);
  const NormArgs<T, P> a = norm_args<T, P>(j);
  const bool even = j.D % V == 0 && norm_rows16<T>(j.x, j.xs, j.N) && norm_rows16<T>(j.y, j.ys, j.N) && on16(j.w) && on16(j.b);
  const bool wide = same_offsets<T>(j.x, j.xs, j.y, j.ys, j.N);
  const long long packs = even ? j.D / V : (j.D + 2 * (V - 1)) / V;  // EDGE: at the worst offset
  auto run = [&](auto* gp) {
    using G = std::remove_pointer_t<decltype(gp)>;
    return launch_pdl(norm_forward_kernel<T, P, G>, (unsigned)((j.N + G::ROWS - 1) / G::ROWS), G::NT, 0, ctx.stream, a);
  };
  auto run_edge = [&](auto* gp) {
    using G = std::remove_pointer_t<decltype(gp)>;
    constexpr int room = 220 * 1024;
    constexpr int row = NormRing<T, G, 1, 1>::STAGE;
    constexpr int rest = 2 * NormParams<P, G>::BYTES + NormRing<T, G, 1, 1>::BYTES - row;
    constexpr int STAGES = (room - rest) / row < 3 ? (room - rest) / row : 3;
    constexpr int smem = STAGES * row + rest;
    static_assert(STAGES >= 1 && smem <= room, "fits");
    auto kernel = norm_forward_edge_kernel<T, P, G, STAGES>;
    const cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    // Two CTAs an SM where their shared memory allows (227 KB, 1 KB of each reserved).
    const long long ctas = smem <= 112 * 1024 && G::NT <= 512 ? 2 : 1;
    return r != cudaSuccess ? r : launch_pdl(kernel, norm_grid(j.N, ctas * ctx.num_sms), G::NT, smem, ctx.stream, a);
  };
  cudaError_t e;
  profile_before(ctx);
  if (even && packs <= 4096 && j.N <= 0x7fffffffll) {
    if (packs <= 32) e = norm_pick<V, 1, 128, false, 32>(packs, run);
    else if (packs <= 64) e = norm_pick<V, 2, 128, false, 32>(packs, run);
    else if (packs <= 128) e = norm_pick<V, 4, 128, false, 32>(packs, run);
    else if (packs <= 256) e = norm_pick<V, 2, 128, false, 128>(packs, run);
    else e = norm_pick<V, 4, 128, false, 96, 128, 192, 256, 384, 512, 768, 1024>(packs, run);
  } else if (wide && packs <= 768 * (16 / V)) {
    constexpr int U = 16 / V;  // 16 values a thread
    e = norm_pick<V, U, 512, true, 32, 64, 96, 128, 192, 256, 384, 512, 768>(packs, run_edge);
  } else {
    e = launch_pdl(norm_forward_long_kernel<T, P>, norm_grid(j.N, 4ll * ctx.num_sms), kNormLongThreads, 0, ctx.stream, a);
  }
  profile_after(ctx);
  return e;
}

template <class T, class P> cudaError_t launch_layer_norm_backward(const LayerNormJob& j, const LaunchCtx& ctx) {
  constexpr int V = 16 / sizeof(T);
  NormArgs<T, P> a = norm_args<T, P>(j);
  const bool sums = j.dw || j.db;
  a.part = sums ? (float*)j.temp : nullptr;
  const bool even = j.D % V == 0 && norm_rows16<T>(j.x, j.xs, j.N) && norm_rows16<T>(j.dy, j.dys, j.N) &&
                    norm_rows16<T>(j.dx, j.dxs, j.N) && on16(j.w);
  const bool wide = same_offsets<T>(j.x, j.xs, j.dy, j.dys, j.N) && same_offsets<T>(j.x, j.xs, j.dx, j.dxs, j.N);
  const long long packs = even ? j.D / V : (j.D + 2 * (V - 1)) / V;
  long long most = ctx.num_sms / 8 * 8;
  if (most > kNormMaxParts) most = kNormMaxParts;
  if (most < 8) most = 8;
  int count = 0;
  auto run = [&](auto* gp) {
    using G = std::remove_pointer_t<decltype(gp)>;
    constexpr int smem = NormBackwardSmem<T, P, G>::BYTES;
    auto kernel = norm_backward_kernel<T, P, G>;
    const cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    const unsigned grid = norm_grid(j.N, most);
    count = (int)grid;
    return r != cudaSuccess ? r : launch_pdl(kernel, grid, G::NT, smem, ctx.stream, a);
  };
  cudaError_t e;
  profile_before(ctx);
  constexpr int U = 16 / V;  // 16 values a thread
  if (even && packs <= 512 * U) {
    e = norm_pick<V, U, 512, false, 32, 64, 96, 128, 192, 256, 384, 512>(packs, run);
  } else if (even && packs <= 512 * 2 * U) {
    e = norm_pick<V, 2 * U, 512, false, 384, 512>(packs, run);
  } else if (wide && packs <= 768 * U) {
    e = norm_pick<V, U, 512, true, 32, 64, 96, 128, 192, 256, 384, 512, 768>(packs, run);
  } else {
    e = launch_pdl(norm_backward_long_kernel<T, P>, norm_grid(j.N, 4ll * ctx.num_sms), kNormLongThreads, 0, ctx.stream, a);
    if (e == cudaSuccess && sums) {
      const long long blocks = (j.D + 255) / 256;
      long long ranges = (8ll * ctx.num_sms + blocks - 1) / blocks;
      if (ranges > j.N) ranges = j.N;
      if (ranges > kNormMaxParts) ranges = kNormMaxParts;
      count = (int)ranges;
      e = launch_pdl(norm_columns_long_kernel<T, P>, (unsigned)(blocks * ranges), 256, 0, ctx.stream, a, count);
    }
  }
  if (e == cudaSuccess && sums)
    e = launch_pdl(norm_fold_kernel<P>, (unsigned)((2 * j.D + 31) / 32), 512, 0, ctx.stream, (const float*)j.temp,
                   count, (int)j.D, (P*)j.dw, (P*)j.db);
  profile_after(ctx);
  return e;
}

}  // namespace gbs
