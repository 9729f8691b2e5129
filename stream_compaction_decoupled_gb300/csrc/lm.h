// lm.h -- host-side interface between the C ABI of the language-model operators
// (lm_api.cu) and their kernel launchers.
#pragma once

#include "launch.h"

namespace gbs {

// A (batch, time, channel) array with unit channel stride: element (b, t, c) is at
// p + b*sb + t*st + c.  p may be null where the array is optional.
struct SeqArray {
  void* p = nullptr;
  long long sb = 0, st = 0;
};

// h_t = a_t h_{t-1} + u_t x_t, a = sigmoid(f), u = sigmoid(i), or 1 - a without i.
struct RecurrenceJob {
  long long B = 0, T = 0, D = 0;
  SeqArray x, f, i, h;              // i.p null: u = 1 - a
  const float* h0 = nullptr;        // (B, D) or null: zero
  const uint8_t* starts = nullptr;  // (B, T) or null: nonzero drops the state before t
  float* last = nullptr;            // forward: (B, D), the state after T steps, or null
  // Backward.
  SeqArray dh, dx, df, di;
  const float* dlast = nullptr;     // (B, D) or null
  float* dh0 = nullptr;             // (B, D) or null
};

// One token for each of B rows against a pool of states.
struct RecurrenceStepJob {
  long long B = 0, D = 0, pool = 0;
  const void *x = nullptr, *f = nullptr, *i = nullptr;
  long long sx = 0, sf = 0, si = 0, sh = 0;  // row strides
  float* state = nullptr;                    // (pool, D)
  const int32_t* slots = nullptr;            // (B) or null: row b uses state b
  void* h = nullptr;
};

// Layer norm of N rows of D values (unit column stride).
struct LayerNormJob {
  long long N = 0, D = 0;
  float eps = 0.f;
  const void* x = nullptr;
  const void* dy = nullptr;  // backward
  void* y = nullptr;         // forward
  void* dx = nullptr;        // backward
  long long xs = 0, dys = 0, ys = 0, dxs = 0;  // row strides
  const void *w = nullptr, *b = nullptr;       // (D) or null
  float *mean = nullptr, *rstd = nullptr;      // (N)
  void *dw = nullptr, *db = nullptr;           // backward: (D) or null
  void* temp = nullptr;                        // backward, with dw or db
};

// The gradient's partial sums over rows: at most this many rows of 2 D floats.
constexpr int kNormMaxParts = 320;
inline size_t layer_norm_temp_bytes(long long N, long long D) {
  const long long parts = N < kNormMaxParts ? (N + 7) / 8 * 8 : kNormMaxParts;
  return round_up((size_t)parts * 2 * (size_t)D * sizeof(float), 256);
}

// Log probabilities of N rows of V logits (unit column stride).
struct LogprobJob {
  long long N = 0, V = 0, stride = 0;
  const void* logits = nullptr;
  const void* targets = nullptr;
  int targets64 = 0;
  float *logprob = nullptr, *entropy = nullptr, *lse = nullptr;  // (N): written, or read by the backward
  int top = 0;
  float* top_values = nullptr;    // (N, top)
  int32_t* top_ids = nullptr;     // (N, top)
  // Backward.
  const float *dlogprob = nullptr, *dentropy = nullptr;  // (N) or null
  void* dlogits = nullptr;
  long long dstride = 0;
};
constexpr int kMaxTop = 32;

template <class T> cudaError_t launch_logprob(const LogprobJob& job, const LaunchCtx& ctx);
template <class T> cudaError_t launch_logprob_backward(const LogprobJob& job, const LaunchCtx& ctx);
template <class T, class P> cudaError_t launch_layer_norm(const LayerNormJob& job, const LaunchCtx& ctx);
template <class T, class P> cudaError_t launch_layer_norm_backward(const LayerNormJob& job, const LaunchCtx& ctx);
template <class T> cudaError_t launch_recurrence(const RecurrenceJob& job, const LaunchCtx& ctx);
template <class T> cudaError_t launch_recurrence_backward(const RecurrenceJob& job, const LaunchCtx& ctx);
template <class T> cudaError_t launch_recurrence_step(const RecurrenceStepJob& job, const LaunchCtx& ctx);

// launch_pdl (launch.h) for a kernel whose CTAs form clusters of `cluster` along x (grid
// a multiple of it).
template <class... P, class... A>
cudaError_t launch_pdl_cluster(void (*kernel)(P...), unsigned grid, unsigned block, unsigned cluster, size_t smem,
                               cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

// How many clusters of the kernel the device can hold at once (-1: the query failed).
template <class... P>
int clusters_resident(void (*kernel)(P...), unsigned block, unsigned cluster, size_t smem) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return -1;
  }
  return n;
}

}  // namespace gbs
