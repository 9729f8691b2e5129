// lm_api.cu -- the C ABI of the language-model operators (declared at the end of
// include/gbscan.h): argument checks and element-type dispatch.  Every check that can
// fail does so before anything is enqueued.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "abi.h"
#include "gbscan.h"
#include "lm.h"

namespace {

using gbs::LaunchCtx;
using gbs::SeqArray;

constexpr long long kMaxLength = 1ll << 30;  // tokens of a sequence, vocabulary
constexpr long long kMaxWidth = 1ll << 28;   // channels, columns: byte offsets within a row fit in 31 bits
constexpr long long kMaxGrid = 0x7fffffffll;

size_t lm_size(int dtype) {
  switch (dtype) {
    case GB_F32: return 4;
    case GB_BF16: case GB_F16: return 2;
    default: return 0;
  }
}

// Calls f with a null pointer to the C++ type of `dtype`.
template <class F> cudaError_t with_lm_type(int dtype, F&& f) {
  switch (dtype) {
    case GB_F32: return f((float*)nullptr);
    case GB_BF16: return f((__nv_bfloat16*)nullptr);
    default: return f((__half*)nullptr);
  }
}
template <class P> using Pointee = std::remove_pointer_t<P>;

bool aligned(const void* p, size_t a) { return (uintptr_t)p % a == 0; }

// Offsets stay within 63 bits.
bool extent_ok(long long n, long long stride) { return n <= 1 || (long double)n * stride < 9.0e17L; }

// Fills `a` from the k-th pair of `strides` (null: contiguous); false if it is not usable.
bool seq(SeqArray& a, const void* p, const int64_t* strides, int k, long long B, long long T, long long D, size_t es) {
  a.p = const_cast<void*>(p);
  a.sb = strides ? strides[2 * k] : T * D;
  a.st = strides ? strides[2 * k + 1] : D;
  return a.sb >= 0 && a.st >= 0 && extent_ok(B, a.sb) && extent_ok(T, a.st) && aligned(p, es);
}

int finish(cudaError_t e) { return e == cudaSuccess ? GB_OK : gbs::abi_cuda_fail(e); }

// The sizes of a recurrence: GB_OK, or what is wrong with them.
int check_sizes(int dtype, long long B, long long T, long long D) {
  if (B < 0 || T < 0 || D < 0) return GB_ERR_INVALID;
  if (!lm_size(dtype)) return GB_ERR_UNSUPPORTED;
  if (D > kMaxWidth || T > kMaxLength || (long double)B * T * D > 9.0e17L) return GB_ERR_RANGE;
  // The narrowest strip is 56 channels, the largest cluster 8 CTAs.
  if ((long double)B * ((D + 31) / 32) * 8 > (long double)kMaxGrid) return GB_ERR_RANGE;
  return GB_OK;
}

}  // namespace

extern "C" {

int gb_recurrence(int dtype, int64_t batch, int64_t length, int64_t channels, const void* x, const void* f,
                  const void* i, const int64_t* strides, const float* h0, const uint8_t* starts, void* h,
                  float* last, void* stream) {
  int rc = check_sizes(dtype, batch, length, channels);
  if (rc) return rc;
  if (batch == 0 || channels == 0 || (length == 0 && !last)) return GB_OK;
  if (length > 0 && (!x || !f || !h)) return GB_ERR_INVALID;
  const size_t es = lm_size(dtype);
  gbs::RecurrenceJob j;
  j.B = batch, j.T = length, j.D = channels;
  if (!seq(j.x, x, strides, 0, batch, length, channels, es) || !seq(j.f, f, strides, 1, batch, length, channels, es) ||
      (i && !seq(j.i, i, strides, 2, batch, length, channels, es)) ||
      !seq(j.h, h, strides, 3, batch, length, channels, es) || !aligned(h0, 4) || !aligned(last, 4))
    return GB_ERR_INVALID;
  j.h0 = h0, j.starts = starts, j.last = last;
  LaunchCtx ctx;
  rc = gbs::abi_ctx(stream, ctx);
  if (rc) return rc;
  return finish(with_lm_type(dtype, [&](auto* tp) { return gbs::launch_recurrence<Pointee<decltype(tp)>>(j, ctx); }));
}

int gb_recurrence_backward(int dtype, int64_t batch, int64_t length, int64_t channels, const void* dh, const void* x,
                           const void* f, const void* i, const void* h, const int64_t* strides, const float* h0,
                           const uint8_t* starts, const float* dlast, void* dx, void* df, void* di, float* dh0,
                           void* stream) {
  int rc = check_sizes(dtype, batch, length, channels);
  if (rc) return rc;
  if (batch == 0 || channels == 0 || (length == 0 && !dh0)) return GB_OK;
  if (length > 0 && (!dh || !x || !f || !h || !dx || !df || (i && !di))) return GB_ERR_INVALID;
  const size_t es = lm_size(dtype);
  gbs::RecurrenceJob j;
  j.B = batch, j.T = length, j.D = channels;
  const auto ok = [&](SeqArray& a, const void* p, int k) { return seq(a, p, strides, k, batch, length, channels, es); };
  if (!ok(j.dh, dh, 0) || !ok(j.x, x, 1) || !ok(j.f, f, 2) || (i && !ok(j.i, i, 3)) || !ok(j.h, h, 4) ||
      !ok(j.dx, dx, 5) || !ok(j.df, df, 6) || (i && !ok(j.di, di, 7)) || !aligned(h0, 4) || !aligned(dlast, 4) ||
      !aligned(dh0, 4))
    return GB_ERR_INVALID;
  j.h0 = h0, j.starts = starts, j.dlast = dlast, j.dh0 = dh0;
  LaunchCtx ctx;
  rc = gbs::abi_ctx(stream, ctx);
  if (rc) return rc;
  return finish(
      with_lm_type(dtype, [&](auto* tp) { return gbs::launch_recurrence_backward<Pointee<decltype(tp)>>(j, ctx); }));
}

int gb_recurrence_step(int dtype, int64_t batch, int64_t channels, const void* x, const void* f, const void* i,
                       const int64_t* strides, float* state, int64_t pool, const int32_t* slots, void* h,
                       void* stream) {
  int rc = check_sizes(dtype, batch, 1, channels);
  if (rc) return rc;
  if (pool < 0) return GB_ERR_INVALID;
  if ((long double)pool * channels > 9.0e17L || (long double)batch * channels > 128.0L * kMaxGrid) return GB_ERR_RANGE;
  if (batch == 0 || channels == 0) return GB_OK;
  if (!x || !f || !h || (pool > 0 && !state)) return GB_ERR_INVALID;
  if (!slots && batch > pool) return GB_ERR_INVALID;
  const size_t es = lm_size(dtype);
  if (!aligned(x, es) || !aligned(f, es) || !aligned(i, es) || !aligned(h, es) || !aligned(state, 4) ||
      !aligned(slots, 4))
    return GB_ERR_INVALID;
  gbs::RecurrenceStepJob j;
  j.B = batch, j.D = channels, j.pool = pool;
  j.x = x, j.f = f, j.i = i, j.h = h, j.state = state, j.slots = slots;
  j.sx = strides ? strides[0] : channels;
  j.sf = strides ? strides[1] : channels;
  j.si = strides ? strides[2] : channels;
  j.sh = strides ? strides[3] : channels;
  for (long long s : {j.sx, j.sf, j.si, j.sh})
    if (s < 0 || !extent_ok(batch, s)) return GB_ERR_INVALID;
  LaunchCtx ctx;
  rc = gbs::abi_ctx(stream, ctx);
  if (rc) return rc;
  return finish(
      with_lm_type(dtype, [&](auto* tp) { return gbs::launch_recurrence_step<Pointee<decltype(tp)>>(j, ctx); }));
}

size_t gb_layer_norm_temp_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || cols > kMaxWidth) return 0;
  return gbs::layer_norm_temp_bytes(rows, cols);
}

int gb_layer_norm(int dtype, int param_dtype, int64_t rows, int64_t cols, const void* x, int64_t x_stride,
                  const void* w, const void* b, float eps, void* y, int64_t y_stride, float* mean, float* rstd,
                  void* stream) {
  if (rows < 0 || cols < 0 || x_stride < 0 || y_stride < 0 || !(eps >= 0.f)) return GB_ERR_INVALID;
  if (!lm_size(dtype) || (param_dtype != dtype && param_dtype != GB_F32)) return GB_ERR_UNSUPPORTED;
  if (cols > kMaxWidth) return GB_ERR_RANGE;
  if (rows == 0 || cols == 0) return GB_OK;
  if (!x || !y || !mean || !rstd) return GB_ERR_INVALID;
  const size_t es = lm_size(dtype), ps = lm_size(param_dtype);
  if (!aligned(x, es) || !aligned(y, es) || !aligned(w, ps) || !aligned(b, ps) || !aligned(mean, 4) ||
      !aligned(rstd, 4) || !extent_ok(rows, x_stride) || !extent_ok(rows, y_stride))
    return GB_ERR_INVALID;
  gbs::LayerNormJob j;
  j.N = rows, j.D = cols, j.eps = eps;
  j.x = x, j.xs = x_stride, j.y = y, j.ys = y_stride, j.w = w, j.b = b, j.mean = mean, j.rstd = rstd;
  LaunchCtx ctx;
  const int rc = gbs::abi_ctx(stream, ctx);
  if (rc) return rc;
  return finish(with_lm_type(dtype, [&](auto* tp) {
    using T = Pointee<decltype(tp)>;
    return param_dtype == dtype ? gbs::launch_layer_norm<T, T>(j, ctx) : gbs::launch_layer_norm<T, float>(j, ctx);
  }));
}

int gb_layer_norm_backward(int dtype, int param_dtype, int64_t rows, int64_t cols, const void* dy, int64_t dy_stride,
                           const void* x, int64_t x_stride, const float* mean, const float* rstd, const void* w,
                           void* dx, int64_t dx_stride, void* dw, void* db, void* temp, size_t temp_bytes,
                           void* stream) {
  if (rows < 0 || cols < 0 || x_stride < 0 || dy_stride < 0 || dx_stride < 0) return GB_ERR_INVALID;
  if (!lm_size(dtype) || (param_dtype != dtype && param_dtype != GB_F32)) return GB_ERR_UNSUPPORTED;
  if (cols > kMaxWidth) return GB_ERR_RANGE;
  if (cols == 0) return GB_OK;
  const size_t es = lm_size(dtype), ps = lm_size(param_dtype);
  if (!aligned(x, es) || !aligned(dy, es) || !aligned(dx, es) || !aligned(w, ps) || !aligned(dw, ps) ||
      !aligned(db, ps) || !aligned(mean, 4) || !aligned(rstd, 4) || !extent_ok(rows, x_stride) ||
      !extent_ok(rows, dy_stride) || !extent_ok(rows, dx_stride))
    return GB_ERR_INVALID;
  if (rows > 0 && (!x || !dy || !dx || !mean || !rstd)) return GB_ERR_INVALID;
  LaunchCtx ctx;
  int rc = gbs::abi_ctx(stream, ctx);
  if (rc) return rc;
  if (rows == 0) {  // the sums over no rows are zero
    cudaError_t e = cudaSuccess;
    if (dw) e = cudaMemsetAsync(dw, 0, (size_t)cols * ps, ctx.stream);
    if (db && e == cudaSuccess) e = cudaMemsetAsync(db, 0, (size_t)cols * ps, ctx.stream);
    return finish(e);
  }
  gbs::LayerNormJob j;
  j.N = rows, j.D = cols;
  j.x = x, j.xs = x_stride, j.dy = dy, j.dys = dy_stride, j.dx = dx, j.dxs = dx_stride;
  j.w = w, j.dw = dw, j.db = db, j.mean = const_cast<float*>(mean), j.rstd = const_cast<float*>(rstd);
  gbs::Temp t;
  if (dw || db) {
    rc = gbs::abi_temp(temp, temp_bytes, gbs::layer_norm_temp_bytes(rows, cols), ctx.stream, t);
    if (rc) return rc;
    j.temp = t.p;
  }
  return finish(with_lm_type(dtype, [&](auto* tp) {
    using T = Pointee<decltype(tp)>;
    return param_dtype == dtype ? gbs::launch_layer_norm_backward<T, T>(j, ctx)
                                : gbs::launch_layer_norm_backward<T, float>(j, ctx);
  }));
}

int gb_token_logprobs(int dtype, int64_t rows, int64_t vocab, const void* logits, int64_t stride, const void* targets,
                      int target_dtype, float* logprob, float* entropy, float* lse, int top, float* top_values,
                      int32_t* top_ids, void* stream) {
  if (rows < 0 || vocab < 0 || stride < 0 || top < 0 || top > gbs::kMaxTop || top > vocab) return GB_ERR_INVALID;
  if (target_dtype != GB_I32 && target_dtype != GB_I64) return GB_ERR_INVALID;
  if (!lm_size(dtype)) return GB_ERR_UNSUPPORTED;
  if (vocab > kMaxLength || rows > kMaxGrid / 8) return GB_ERR_RANGE;
  if (rows == 0) return GB_OK;
  if ((vocab > 0 && !logits) || !targets || !logprob || !entropy || !lse) return GB_ERR_INVALID;
  if (top > 0 && (!top_values || !top_ids)) return GB_ERR_INVALID;
  if (!aligned(logits, lm_size(dtype)) || !aligned(targets, target_dtype == GB_I64 ? 8 : 4) || !aligned(logprob, 4) ||
      !aligned(entropy, 4) || !aligned(lse, 4) || !aligned(top_values, 4) || !aligned(top_ids, 4) ||
      !extent_ok(rows, stride))
    return GB_ERR_INVALID;
  gbs::LogprobJob j;
  j.N = rows, j.V = vocab, j.stride = stride, j.logits = logits, j.targets = targets;
  j.targets64 = target_dtype == GB_I64;
  j.logprob = logprob, j.entropy = entropy, j.lse = lse;
  j.top = top, j.top_values = top_values, j.top_ids = top_ids;
  LaunchCtx ctx;
  const int rc = gbs::abi_ctx(stream, ctx);
  if (rc) return rc;
  return finish(with_lm_type(dtype, [&](auto* tp) { return gbs::launch_logprob<Pointee<decltype(tp)>>(j, ctx); }));
}

int gb_token_logprobs_backward(int dtype, int64_t rows, int64_t vocab, const void* logits, int64_t stride,
                               const void* targets, int target_dtype, const float* lse, const float* entropy,
                               const float* dlogprob, const float* dentropy, void* dlogits, int64_t dstride,
                               void* stream) {
  if (rows < 0 || vocab < 0 || stride < 0 || dstride < 0) return GB_ERR_INVALID;
  if (target_dtype != GB_I32 && target_dtype != GB_I64) return GB_ERR_INVALID;
  if (!lm_size(dtype)) return GB_ERR_UNSUPPORTED;
  // The narrowest block of a row is 1024 values.
  if (vocab > kMaxLength || (long double)rows * ((vocab + 1023) / 1024) > (long double)kMaxGrid) return GB_ERR_RANGE;
  if (rows == 0 || vocab == 0) return GB_OK;
  if (!logits || !targets || !lse || !dlogits || (dentropy && !entropy)) return GB_ERR_INVALID;
  if (logits == dlogits && stride != dstride) return GB_ERR_INVALID;
  const size_t es = lm_size(dtype);
  if (!aligned(logits, es) || !aligned(dlogits, es) || !aligned(targets, target_dtype == GB_I64 ? 8 : 4) ||
      !aligned(lse, 4) || !aligned(entropy, 4) || !aligned(dlogprob, 4) || !aligned(dentropy, 4) ||
      !extent_ok(rows, stride) || !extent_ok(rows, dstride))
    return GB_ERR_INVALID;
  gbs::LogprobJob j;
  j.N = rows, j.V = vocab, j.stride = stride, j.logits = logits, j.targets = targets;
  j.targets64 = target_dtype == GB_I64;
  j.lse = const_cast<float*>(lse), j.entropy = const_cast<float*>(entropy);
  j.dlogprob = dlogprob, j.dentropy = dentropy, j.dlogits = dlogits, j.dstride = dstride;
  LaunchCtx ctx;
  const int rc = gbs::abi_ctx(stream, ctx);
  if (rc) return rc;
  return finish(
      with_lm_type(dtype, [&](auto* tp) { return gbs::launch_logprob_backward<Pointee<decltype(tp)>>(j, ctx); }));
}

}  // extern "C"
