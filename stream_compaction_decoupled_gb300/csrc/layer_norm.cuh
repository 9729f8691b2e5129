// layer_norm.cuh -- layer norm over the rows of a matrix and its gradient.
//
//   mean = sum x / D,  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps),  n = (x - mean) rstd,
//   y = n w + b;
//   g = dy w:  dx = rstd (g - mean(g) - n mean(g n)),   dw = sum_rows dy n,  db = sum_rows dy.
//
// A row is held in the registers of TPR threads, so it is read once: the mean first, then
// the centred squares (no cancellation), then y.  CTAs are persistent: CTA c takes rows
// c + G k (G the grid, a multiple of 8), which has two uses.  The weight is loaded once a
// CTA, and the gradient's sums over rows stay in registers until the CTA is done; one row
// of partial sums a CTA is then reduced by a second, small launch, in a fixed order.  And
// every row of a CTA starts at the same offset from a 16-byte boundary, whatever the width
// (the offset repeats after at most 8 rows), so an odd width is read in whole 16-byte
// packs too: the packs are laid over the row shifted by the offset, and only the first
// and the last of a row are read value by value.
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
template <int V_, int TPR_, int NV_> struct NormGeom {
  static constexpr int V = V_, TPR = TPR_, NV = NV_;
  static constexpr int NT = TPR < 256 ? 256 : TPR;
  static constexpr int ROWS = NT / TPR;       // rows a CTA takes at a time
  static constexpr int WARPS = TPR / 32;      // warps of a row
  // Whether the weight (and in the forward pass the next row, in the backward the row
  // between its two passes) is held in registers.  At 32 values a thread there is no room:
  // what is needed is read again, from L1 or L2.
  static constexpr bool HOLD = NV * V <= 16;
  // Where the gradient's sums over rows are kept: in registers, or, at 512 threads a row
  // (128 registers a thread at most), in shared memory, each thread's own.
  static constexpr bool SUMS_IN_SMEM = TPR >= 512;
  static constexpr size_t SUMS_BYTES = SUMS_IN_SMEM ? (size_t)NT * NV * V * 2 * sizeof(float) : 0;
};

// Values e0 .. e0 + V - 1 of a row of D values, the first of them at p; those outside the
// row read as zero and are not written.
template <class T, int V> __device__ __forceinline__ Pack<T, V> norm_load(const T* p, int e0, int D, bool on) {
  Pack<T, V> r;
  if (on && e0 >= 0 && e0 + V <= D) {
    r = ld_pack<T, V>(p);
  } else {
#pragma unroll
    for (int c = 0; c < V; ++c) r.v[c] = on && (unsigned)(e0 + c) < (unsigned)D ? p[c] : narrow<T>(0.f);
  }
  return r;
}
template <class T, int V> __device__ __forceinline__ void norm_store(T* p, int e0, int D, const Pack<T, V>& v) {
  if (e0 >= 0 && e0 + V <= D) {
    st_pack(p, v);
  } else {
#pragma unroll
    for (int c = 0; c < V; ++c)
      if ((unsigned)(e0 + c) < (unsigned)D) p[c] = v.v[c];
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
    __syncthreads();
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

template <class T, class P, class G>
__global__ void __launch_bounds__(G::NT) norm_forward_kernel(const __grid_constant__ NormArgs<T, P> a) {
  constexpr int V = G::V, NV = G::NV;
  __shared__ NormShared<G> sh;
  pdl_entry();
  const int t = threadIdx.x % G::TPR, sub = threadIdx.x / G::TPR;
  const long long first = blockIdx.x;
  if (first >= a.N) return;
  const int off = (int)((uintptr_t)(a.x + first * a.xs) % 16 / sizeof(T));
  const int e0 = t * V - off;  // this thread's first value; its packs are kStep apart
  constexpr int kStep = G::TPR * V;
  P w[NV][V], b[NV][V];
  auto affine = [&](int i) {
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const int e = e0 + i * kStep + c;
      const bool in = (unsigned)e < (unsigned)a.D;
      w[i][c] = in && a.w ? a.w[e] : narrow<P>(1.f);
      b[i][c] = in && a.b ? a.b[e] : narrow<P>(0.f);
    }
  };
  if constexpr (G::HOLD) {
#pragma unroll
    for (int i = 0; i < NV; ++i) affine(i);
  }
  const float inv = 1.f / (float)a.D;
  int turn = 0;
  Pack<T, V> px[NV];
  auto load = [&](long long row) {
    const T* p = a.x + row * a.xs + e0;
#pragma unroll
    for (int i = 0; i < NV; ++i) px[i] = norm_load<T, V>(p + i * kStep, e0 + i * kStep, a.D, row < a.N);
  };
  const long long G_ = gridDim.x;
  if constexpr (G::HOLD) load(first + G_ * sub);
  for (long long base = first; base < a.N; base += G_ * G::ROWS) {
    const long long row = base + G_ * sub;
    const bool live = row < a.N;
    float x[NV][V];
    if constexpr (!G::HOLD) load(row);
#pragma unroll
    for (int i = 0; i < NV; ++i) widen_pack(px[i], x[i]);
    if constexpr (G::HOLD) load(row + G_ * G::ROWS);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int c = 0; c < V; ++c) s += x[i][c];
    const float mean = norm_sum<G>(make_float2(s, 0.f), sh, turn).x * inv;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int c = 0; c < V; ++c) {
        x[i][c] = (unsigned)(e0 + i * kStep + c) < (unsigned)a.D ? x[i][c] - mean : 0.f;
        q = fmaf(x[i][c], x[i][c], q);
      }
    const float var = norm_sum<G>(make_float2(q, 0.f), sh, turn).x * inv;
    const float rstd = 1.f / sqrtf(var + a.eps);
    if (!live) continue;
    if (t == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (!G::HOLD) affine(i);
#pragma unroll
      for (int c = 0; c < V; ++c) x[i][c] = fmaf(x[i][c] * rstd, widen(w[i][c]), widen(b[i][c]));
      norm_store<T, V>(a.y + row * a.ys + e0 + i * kStep, e0 + i * kStep, a.D, narrow_pack<T, V>(x[i]));
    }
  }
}

template <class T, class P, class G>
__global__ void __launch_bounds__(G::NT) norm_backward_kernel(const __grid_constant__ NormArgs<T, P> a) {
  constexpr int V = G::V, NV = G::NV;
  constexpr int kSums = G::SUMS_IN_SMEM ? 1 : NV * V;
  __shared__ NormShared<G> sh;
  __shared__ float fold[G::ROWS > 1 ? G::NT * NV * V : 1];
  extern __shared__ float sums_mem[];
  pdl_entry();
  const int t = threadIdx.x % G::TPR, sub = threadIdx.x / G::TPR;
  const long long first = blockIdx.x;
  const int off = first < a.N ? (int)((uintptr_t)(a.x + first * a.xs) % 16 / sizeof(T)) : 0;
  const int e0 = t * V - off;
  constexpr int kStep = G::TPR * V;
  float dw_[kSums], db_[kSums];
  auto dw = [&](int k) -> float& {
    if constexpr (G::SUMS_IN_SMEM) return sums_mem[k * G::NT + threadIdx.x];
    else return dw_[k];
  };
  auto db = [&](int k) -> float& {
    if constexpr (G::SUMS_IN_SMEM) return sums_mem[(NV * V + k) * G::NT + threadIdx.x];
    else return db_[k];
  };
  constexpr int kHeld = G::HOLD ? NV : 1;
  P pw[kHeld][V];
  auto weight = [&](int i) {
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const int e = e0 + i * kStep + c;
      pw[i % kHeld][c] = a.w && (unsigned)e < (unsigned)a.D ? a.w[e] : narrow<P>(1.f);
    }
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int c = 0; c < V; ++c) dw(i * V + c) = db(i * V + c) = 0.f;
    if constexpr (G::HOLD) weight(i);
  }
  const float inv = 1.f / (float)a.D;
  int turn = 0;
  const long long G_ = gridDim.x;
  for (long long base = first; base < a.N; base += G_ * G::ROWS) {
    const long long row = base + G_ * sub;
    const bool live = row < a.N;
    const T *x_at = a.x + row * a.xs + e0, *dy_at = a.dy + row * a.dys + e0;
    Pack<T, V> px[kHeld], pd[kHeld];
    auto load = [&](int i) {
      px[i % kHeld] = norm_load<T, V>(x_at + i * kStep, e0 + i * kStep, a.D, live);
      pd[i % kHeld] = norm_load<T, V>(dy_at + i * kStep, e0 + i * kStep, a.D, live);
    };
    if constexpr (G::HOLD) {
#pragma unroll
      for (int i = 0; i < NV; ++i) load(i);
    }
    const float mean = live ? a.mean[row] : 0.f, rstd = live ? a.rstd[row] : 0.f;
    float2 s = make_float2(0.f, 0.f);
#pragma unroll kHeld
    for (int i = 0; i < NV; ++i) {
      float x[V], d[V];
      if constexpr (!G::HOLD) load(i), weight(i);
      widen_pack(px[i % kHeld], x);
      widen_pack(pd[i % kHeld], d);  // zero outside the row
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float n = (x[c] - mean) * rstd;
        dw(i * V + c) = fmaf(d[c], n, dw(i * V + c));
        db(i * V + c) += d[c];
        const float g = d[c] * widen(pw[i % kHeld][c]);
        s.x += g;
        s.y = fmaf(g, n, s.y);
      }
    }
    s = norm_sum<G>(s, sh, turn);
    const float mg = s.x * inv, mgn = s.y * inv;
    if (!live) continue;
#pragma unroll kHeld
    for (int i = 0; i < NV; ++i) {
      float x[V], d[V];
      if constexpr (!G::HOLD) load(i), weight(i);
      widen_pack(px[i % kHeld], x);
      widen_pack(pd[i % kHeld], d);
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float n = (x[c] - mean) * rstd;
        d[c] = (fmaf(-n, mgn, d[c] * widen(pw[i % kHeld][c])) - mg) * rstd;
      }
      norm_store<T, V>(a.dx + row * a.dxs + e0 + i * kStep, e0 + i * kStep, a.D, narrow_pack<T, V>(d));
    }
  }
  if (!a.part) return;
  float* part = a.part + (size_t)blockIdx.x * 2 * a.D;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
#pragma unroll
    for (int k = 0; k < NV * V; ++k) {
      const float v = which ? db(k) : dw(k);
      const int e = e0 + k / V * kStep + k % V;
      if constexpr (G::ROWS > 1) fold[k * G::NT + threadIdx.x] = v;
      else if ((unsigned)e < (unsigned)a.D) part[(size_t)which * a.D + e] = v;
    }
    if constexpr (G::ROWS > 1) {
      __syncthreads();
      if (sub == 0) {
#pragma unroll
        for (int k = 0; k < NV * V; ++k) {
          float v = 0.f;
#pragma unroll
          for (int r = 0; r < G::ROWS; ++r) v += fold[k * G::NT + r * G::TPR + t];
          const int e = e0 + k / V * kStep + k % V;
          if ((unsigned)e < (unsigned)a.D) part[(size_t)which * a.D + e] = v;
        }
      }
      __syncthreads();
    }
  }
}

// Rows of any alignment and length, value by value: the row is read again for each of
// the passes (from L2).  Rows too long for registers, and arrays whose rows start at
// different offsets from a 16-byte boundary, come here.
constexpr int kNormLongThreads = 512;
using NormLongGeom = NormGeom<1, kNormLongThreads, 1>;

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

// dw and db from `count` rows of partial sums: 32 columns a CTA, 8 threads a column.
template <class P>
__global__ void __launch_bounds__(256) norm_fold_kernel(const float* part, int count, int D, P* dw, P* db) {
  __shared__ float red[8][33];
  pdl_entry();
  const int lane = threadIdx.x % 32, g = threadIdx.x / 32;
  const int at = blockIdx.x * 32 + lane;  // a column of (dw, db) side by side
  float s = 0.f;
  if (at < 2 * D) {
#pragma unroll 8
    for (int p = g; p < count; p += 8) s += part[(size_t)p * 2 * D + at];
  }
  red[g][lane] = s;
  __syncthreads();
  if (g == 0 && at < 2 * D) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += red[k][lane];
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

// Calls f(geometry) with the first geometry that holds a row of D values at any offset,
// or f(nullptr) where none does.
template <class T, class F> cudaError_t norm_geometry(long long D, F&& f) {
  constexpr int V = 16 / sizeof(T);
  const long long packs = (D + 2 * (V - 1)) / V;  // at the worst offset
  if (packs <= 32 * (8 / V)) return f((NormGeom<V, 32, 8 / V>*)nullptr);
  if (packs <= 32 * (16 / V)) return f((NormGeom<V, 32, 16 / V>*)nullptr);
  if (packs <= 128 * (16 / V)) return f((NormGeom<V, 128, 16 / V>*)nullptr);
  if (packs <= 256 * (16 / V)) return f((NormGeom<V, 256, 16 / V>*)nullptr);
  if (packs <= 512 * (16 / V)) return f((NormGeom<V, 512, 16 / V>*)nullptr);
  if (packs <= 512 * (32 / V)) return f((NormGeom<V, 512, 32 / V>*)nullptr);
  return f((void*)nullptr);
}

// CTAs: enough for every row, at most `most`; a multiple of 8 (see the top of the file).
inline unsigned norm_grid(long long N, int rows, long long most) {
  long long g = (N + rows - 1) / rows;
  if (g > most) g = most;
  return (unsigned)((g + 7) / 8 * 8);
}

template <class T, class P> cudaError_t launch_layer_norm(const LayerNormJob& j, const LaunchCtx& ctx) {
  const NormArgs<T, P> a = norm_args<T, P>(j);
  profile_before(ctx);
  const bool wide = same_offsets<T>(j.x, j.xs, j.y, j.ys, j.N);
  cudaError_t e = norm_geometry<T>(wide ? j.D : 0x7fffffff, [&](auto* gp) {
    using G = std::remove_pointer_t<decltype(gp)>;
    if constexpr (std::is_void_v<G>)
      return launch_pdl(norm_forward_long_kernel<T, P>, norm_grid(j.N, 1, 4ll * ctx.num_sms), kNormLongThreads, 0,
                        ctx.stream, a);
    else
      return launch_pdl(norm_forward_kernel<T, P, G>, norm_grid(j.N, G::ROWS, 1024ll / G::NT * ctx.num_sms), G::NT, 0,
                        ctx.stream, a);
  });
  profile_after(ctx);
  return e;
}

template <class T, class P> cudaError_t launch_layer_norm_backward(const LayerNormJob& j, const LaunchCtx& ctx) {
  NormArgs<T, P> a = norm_args<T, P>(j);
  const bool sums = j.dw || j.db;
  a.part = sums ? (float*)j.temp : nullptr;
  int count = 0;
  profile_before(ctx);
  const bool wide = same_offsets<T>(j.x, j.xs, j.dy, j.dys, j.N) && same_offsets<T>(j.x, j.xs, j.dx, j.dxs, j.N);
  cudaError_t e = norm_geometry<T>(wide ? j.D : 0x7fffffff, [&](auto* gp) {
    using G = std::remove_pointer_t<decltype(gp)>;
    if constexpr (std::is_void_v<G>) {
      cudaError_t r = launch_pdl(norm_backward_long_kernel<T, P>, norm_grid(j.N, 1, 4ll * ctx.num_sms),
                                 kNormLongThreads, 0, ctx.stream, a);
      if (r != cudaSuccess || !sums) return r;
      const long long blocks = (j.D + 255) / 256;
      long long ranges = (8ll * ctx.num_sms + blocks - 1) / blocks;
      if (ranges > j.N) ranges = j.N;
      if (ranges > kNormMaxParts) ranges = kNormMaxParts;
      count = (int)ranges;
      return launch_pdl(norm_columns_long_kernel<T, P>, (unsigned)(blocks * ranges), 256, 0, ctx.stream, a, count);
    } else {
      long long most = 512ll / G::NT * ctx.num_sms;
      if (most > kNormMaxParts) most = kNormMaxParts;
      const unsigned grid = norm_grid(j.N, G::ROWS, most / 8 * 8);
      count = (int)grid;
      auto kernel = norm_backward_kernel<T, P, G>;
      cudaError_t r = cudaSuccess;
      if (G::SUMS_BYTES)
        r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)G::SUMS_BYTES);
      return r != cudaSuccess ? r : launch_pdl(kernel, grid, G::NT, G::SUMS_BYTES, ctx.stream, a);
    }
  });
  if (e == cudaSuccess && sums)
    e = launch_pdl(norm_fold_kernel<P>, (unsigned)((2 * j.D + 31) / 32), 256, 0, ctx.stream, (const float*)j.temp,
                   count, (int)j.D, (P*)j.dw, (P*)j.db);
  profile_after(ctx);
  return e;
}

}  // namespace gbs
