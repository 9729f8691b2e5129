// lm.cuh -- device helpers of the language-model operators (recurrence, layer norm, token
// log probabilities, causal convolution, selective scan, verification of drafts): 16-byte
// vectors of fp32 / bf16 / fp16 values widened to fp32, the approximate exponential and
// reciprocal, sigmoid and softplus, asynchronous copies into shared memory, thread-block
// clusters.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace gbs {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLn2Low = (float)(0.6931471805599453 - (double)kLn2);  // ln 2 is the two's sum

// ---- element types: all arithmetic is in fp32, each output is rounded once ----------

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float widen(__half v) { return __half2float(v); }
template <class T> __device__ __forceinline__ T narrow(float v);
template <> __device__ __forceinline__ float narrow<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half narrow<__half>(float v) { return __float2half_rn(v); }

// V consecutive values (V = 1, or 16 bytes' worth) as they lie in memory.
template <class T, int V> struct Pack {
  static_assert(V == 1 || V * sizeof(T) == 16, "one value or 16 bytes");
  alignas(V == 1 ? sizeof(T) : 16) T v[V];
};
template <class T, int V> __device__ __forceinline__ Pack<T, V> ld_pack(const T* p) {
  Pack<T, V> r;
  if constexpr (V == 1) {
    r.v[0] = *p;
  } else {
    const uint4 u = *(const uint4*)p;
    memcpy(r.v, &u, 16);
  }
  return r;
}
template <class T, int V> __device__ __forceinline__ void st_pack(T* p, const Pack<T, V>& x) {
  if constexpr (V == 1) {
    *p = x.v[0];
  } else {
    uint4 u;
    memcpy(&u, x.v, 16);
    *(uint4*)p = u;
  }
}
// Two 16-bit values in a register, as they lie in memory, to and from fp32: one or two
// instructions a pair (a bf16 is the upper half of an fp32).
template <class T> __device__ __forceinline__ float2 widen2(unsigned w);
template <> __device__ __forceinline__ float2 widen2<__nv_bfloat16>(unsigned w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 widen2<__half>(unsigned w) {
  __half2 h;
  memcpy(&h, &w, 4);
  return __half22float2(h);
}
template <class T> __device__ __forceinline__ unsigned narrow2(float2 v);
template <> __device__ __forceinline__ unsigned narrow2<__nv_bfloat16>(float2 v) {
  unsigned w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(v.y), "f"(v.x));
  return w;
}
template <> __device__ __forceinline__ unsigned narrow2<__half>(float2 v) {
  unsigned w;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(v.y), "f"(v.x));
  return w;
}
template <class T, int V> __device__ __forceinline__ void widen_pack(const Pack<T, V>& x, float (&f)[V]) {
  if constexpr (V == 8) {
    unsigned w[4];
    memcpy(w, &x, 16);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 q = widen2<T>(w[k]);
      f[2 * k] = q.x;
      f[2 * k + 1] = q.y;
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = widen(x.v[k]);
  }
}
template <class T, int V> __device__ __forceinline__ Pack<T, V> narrow_pack(const float (&f)[V]) {
  Pack<T, V> r;
  if constexpr (V == 8) {
    unsigned w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = narrow2<T>(make_float2(f[2 * k], f[2 * k + 1]));
    memcpy(&r, w, 16);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) r.v[k] = narrow<T>(f[k]);
  }
  return r;
}

// ---- approximate functions (PTX instructions) -----------------------------------------
// The instructions are off by a few units in the last place (ex2: 2.5 units of 2^-24 measured).
// A function whose argument was rounded first is off by more: 2^(x log2(e)) by 0.7 |x log2(e)|
// units of 2^-24 besides.


__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 operations in one instruction (sm_100 and later).  The assembler fuses a product
// into a sum that follows it (measured: add2(mul2(a, b), c) has the bits of fma2(a, b, c)) in
// one place and not in another: where bits must be the same, no sum takes a product.
__device__ __forceinline__ unsigned long long bits2(float2 v) {
  unsigned long long u;
  asm("mov.b64 %0, {%1, %2};" : "=l"(u) : "f"(v.x), "f"(v.y));
  return u;
}
__device__ __forceinline__ float2 float2_of(unsigned long long u) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(u));
  return v;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return float2_of(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(d);
}
// e^d to 4 units of 2^-24, for finite d: 2^y, y = d log2(e) rounded, and what that rounding lost,
// e^(d - y ln 2) = 1 + (d - y ln 2).
__device__ __forceinline__ float2 exp_full(float2 d) {
  const float2 y = mul2(d, make_float2(kLog2e, kLog2e)), e = make_float2(ex2(y.x), ex2(y.y));
  const float2 lost = fma2(y, make_float2(-kLn2Low, -kLn2Low), fma2(y, make_float2(-kLn2, -kLn2), d));
  return fma2(e, lost, e);
}
// min / max that keep a NaN operand (fminf and fmaxf drop it).
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

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

// log(1 + e^v) = max(v, 0) + log(1 + e^-|v|) of two values, relatively accurate where it is small:
// log(1 + e) / e on [0, 1] is a polynomial of least relative error (exchange algorithm in 64 bits; off by
// 2.6 units of 2^-24 in fp32 arithmetic).
__device__ __forceinline__ float2 softplus2(float2 v) {
  constexpr float c[] = {1.f, -0.499999017f, 0.333299637f, -0.249541342f, 0.196759388f, -0.153055921f,
                         0.106036551f, -0.0569595359f, 0.0198514629f, -0.00324402517f};
  const float2 e = exp_full(make_float2(fmaxf(-fabsf(v.x), -104.f), fmaxf(-fabsf(v.y), -104.f)));
  float2 p = make_float2(c[9], c[9]);
#pragma unroll
  for (int k = 8; k >= 0; --k) p = fma2(p, e, make_float2(c[k], c[k]));
  return fma2(e, p, make_float2(max_nan(v.x, 0.f), max_nan(v.y, 0.f)));
}

// ---- asynchronous copies of 16 bytes, tracked by the issuing thread ------------------

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// Copies the first `bytes` (1 .. 16) of 16 bytes and writes zeros for the rest.
__device__ __forceinline__ void cp_async_part(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---- clusters ------------------------------------------------------------------------

// All threads of all CTAs of the cluster: what was written before the barrier, in any of
// their shared memories, is visible after it.  A hardware barrier over CTAs that the GPU
// schedules together, not a spin.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same barrier without the order of memory: no fence behind this CTA's stores.  The
// threads of a warp need not come together.
__device__ __forceinline__ void cluster_sync_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  asm volatile("barrier.cluster.wait;" ::: "memory");
}
__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The shared-memory address, in CTA `rank` of the cluster, of the variable at `p` here.
__device__ __forceinline__ unsigned cluster_addr(const void* p, unsigned rank) {
  unsigned a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
// Stores 16 bytes in another CTA's shared memory and counts them on an mbarrier there.
__device__ __forceinline__ void st_async_f4(unsigned addr, float4 v, unsigned bar) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
      "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)), "r"(__float_as_uint(v.z)), "r"(__float_as_uint(v.w)),
      "r"(bar)
      : "memory");
}
// Waits, for at most limit_ns of global time, for phase `parity` of an mbarrier that such
// stores complete.  The acquire is at cluster scope: the data comes from other CTAs.
__device__ __forceinline__ bool mbar_try_wait_cluster(unsigned long long* bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_cluster(unsigned long long* bar, unsigned parity, unsigned long long limit_ns) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const unsigned long long t0 = globaltimer();
  while (!mbar_try_wait_cluster(bar, parity)) {
    if (globaltimer() - t0 > limit_ns) return false;
  }
  return true;
}
__device__ __forceinline__ float ld_cluster_f32(unsigned addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ unsigned long long ld_cluster_u64(unsigned addr) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

}  // namespace gbs
