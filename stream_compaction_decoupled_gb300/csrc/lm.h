// lm.h -- host-side interface between the C ABI of the language-model operators
// (lm_api.cu) and their kernel launchers.
#pragma once

#include <math.h>

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

// A short causal convolution of each channel over time:
// y_t = act(bias + sum_k w_k x_{t-taps+1+k}), act silu or the identity.
struct CausalConvJob {
  long long B = 0, T = 0, D = 0;
  int taps = 0, silu = 0, wide_params = 0;  // wide_params: w and bias (dw and db) are fp32
  SeqArray x, y;
  const void *w = nullptr, *bias = nullptr;  // (D, taps), (D) or null
  const void* state = nullptr;               // (B, taps - 1, D) or null: zero
  const uint8_t* starts = nullptr;           // (B, T) or null
  void* last = nullptr;                      // (B, taps - 1, D) or null
  // Backward.
  SeqArray dy, dx;
  const void* dlast = nullptr;               // (B, taps - 1, D) or null
  void *dw = nullptr, *db = nullptr;         // like w, bias, or null
  void* dstate = nullptr;                    // (B, taps - 1, D) or null
  void* temp = nullptr;                      // with dw or db
};
constexpr int kConvMaxTaps = 8;
// How the gradient splits its tokens: a warp takes a run of `length` tokens of every slots-th
// batch row, and leaves a row of partial sums for the weights.
struct ConvSplit {
  long long slots, runs, length;
};
// warps: how many run on an SM at once.  More of them give more runs: the scratch is sized for 12.
inline ConvSplit conv_backward_split(long long B, long long T, long long D, int warps) {
  long long want = 152 * warps / ((D + 127) / 128);  // of 128 channels
  if (want < 1) want = 1;
  const long long per_row = want / B > 1 ? want / B : 1;
  long long length = (T + per_row - 1) / per_row;
  length = length < 32 ? 32 : (length + 7) / 8 * 8;  // a run reads up to 14 tokens of its neighbours
  const long long runs = (T + length - 1) / length;
  return {B < 4 * want ? B : 4 * want, runs < 1 ? 1 : runs, length};
}
inline size_t conv_temp_bytes(long long B, long long T, long long D, int taps) {
  const ConvSplit s = conv_backward_split(B, T, D, 12);
  return round_up((size_t)(s.slots * s.runs) * (taps + 1) * (size_t)D * sizeof(float), 256);
}

struct CausalConvStepJob {
  long long B = 0, D = 0, pool = 0;
  int taps = 0, silu = 0, wide_params = 0;
  const void *x = nullptr, *w = nullptr, *bias = nullptr;
  long long sx = 0, sy = 0;        // row strides
  void* state = nullptr;           // (pool, taps - 1, D)
  const int32_t* slots = nullptr;  // (B) or null: row b uses state b
  void* y = nullptr;
};

// A (batch, time, group, state) array with unit state stride.
struct GroupArray {
  void* p = nullptr;
  long long sb = 0, st = 0, sg = 0;
};

// h_t = exp(D_t A) h_{t-1} + D_t x_t B_t, y_t = (C_t . h_t + d x_t) silu(z_t),
// D_t = softplus(dt_t + bias) or dt_t + bias: N states a channel, channels in G groups that
// share B and C.
struct SelectiveScanJob {
  long long B = 0, T = 0, D = 0, N = 0, G = 0;
  int softplus = 0;
  SeqArray x, dt, z, y;                // z.p null: no gate
  GroupArray b, c;
  const float *a = nullptr;            // (D, N)
  const float *d = nullptr, *bias = nullptr;  // (D) or null
  const float* h0 = nullptr;           // (B, D, N) or null: zero
  const uint8_t* starts = nullptr;     // (B, T) or null
  float* last = nullptr;               // (B, D, N) or null
  float* kept = nullptr;               // (B, ceil(T / 16), D, N) or null; the backward reads it
  // Backward.
  SeqArray dy, dx, ddt, dz;
  GroupArray db, dc;
  const float* dlast = nullptr;        // (B, D, N) or null
  float *da = nullptr, *dd = nullptr, *dbias = nullptr;  // (D, N), (D), (D); the last two may be null
  float* dh0 = nullptr;                // (B, D, N) or null
  void* temp = nullptr;
};
constexpr int kSscTile = 16;      // tokens of a tile: a kept state precedes each
constexpr int kSscChannels = 64;  // channels of a block
constexpr int kSscMaxStates = 128;
// How the tokens of a batch row are split: parts of `tiles` tiles each, which run side by side.
struct SscSplit {
  long long parts, tiles;
};
constexpr long long kSscSms = 152;  // GB300's: the scratch is sized without asking a device
// Shared memory of a block of 4 warps, states in NB blocks of 16, values of es bytes.
constexpr size_t ssc_forward_bytes(int es, int lanes, int NB) {
  return 4 * (size_t)((es == 2 ? 3 : 2) * (3 * 8 * (64 / lanes) * es + NB * 8 * 32 * es) + NB * 8 * 32 * 4 + 8 * (32 / lanes) * 16 +
                      (NB > 1 ? NB * 16 / lanes * 256 : 0));
}
constexpr size_t ssc_backward_bytes(int es, int NB) {
  return 4 * (size_t)(2 * (4 * 16 * 16 * es + 1024) + 2048 + 1024 + 2 * 3 * 1024 + 2048 + (NB > 1 ? NB * 2048 : 0)) +
         2 * 16 * 32 * es + NB * 2048;
}
// Blocks an SM holds: by registers `bound`, by shared memory what goes into 228 KB (with 1 KB a block of
// the system's).
constexpr int ssc_resident(size_t bytes, int bound) {
  return 228 * 1024 / (bytes + 1024) < (size_t)bound ? (int)(228 * 1024 / (bytes + 1024)) : bound;
}
// What a split costs, in the time that a tile takes a block alone on its SM.  k blocks of an SM take
// 1 + share (k - 1) a tile, and each block `start` tiles' time to begin; the first pass, over all parts but
// the last, takes `again` of that; each part goes through all before it first, `part` for each of them;
// `launch` is the second launch's.
struct SscCost {
  double share, again, part, launch, start;
};
inline double ssc_waves(long long blocks, int resident, double share) {
  const long long most = resident * kSscSms, rest = blocks % most;
  const double all = 1 + share * (resident - 1), last = rest ? 1 + share * (double)((rest - 1) / kSscSms) : 0;
  return (double)(blocks / most) * all + last;
}
// The split that costs least, of those whose blocks are one to 16 for each SM: parts of 2 tiles at least, and
// not so many that the way through the parts before one becomes as long as a part.
// units: blocks, where a row is one part; two waves of them fill the device anyway.
inline SscSplit ssc_best_split(long long tiles, long long units, int resident, const SscCost& c, double& cost) {
  SscSplit best = {1, tiles};
  cost = ((double)tiles + c.start) * ssc_waves(units, resident, c.share);
  if (tiles < 8 || units >= 2 * resident * kSscSms) return best;
  const long long root = (long long)sqrt(8.0 * (double)tiles), most = root < tiles / 2 ? root : tiles / 2;
  for (long long each_sm = 1, tried = 1; each_sm <= 16 && tried < most; ++each_sm) {
    const long long fit = each_sm * kSscSms / units, p = fit < most ? fit : most;
    if (p <= tried) continue;
    tried = p;
    const long long each = (tiles + p - 1) / p, parts = (tiles + each - 1) / each;
    const double waves = ssc_waves(units * parts, resident, c.share) + c.again * ssc_waves(units * (parts - 1), resident, c.share);
    const double x = ((double)each + c.start) * waves + c.part * (double)parts + c.launch;
    if (x < cost) cost = x, best = {parts, each};
  }
  return best;
}
// The gradient: a block takes 64 channels.  (bf16, us: 7 x 2048 x 1024, 16 states, 112 blocks, one part 621, 2
// 519, 8 400; 8 x 2048 x 2048, 256 blocks, one 825, in 4 parts 898; 4 x 1024 x 2048, 128 states, of which a
// block fills an SM, one part 2979, 8 3392.)
inline SscSplit ssc_backward_split(long long B, long long T, long long D, long long N, long long G, int es) {
  const int NB = (int)((N + 15) / 16);
  const long long units = B * G * ((D / G + kSscChannels - 1) / kSscChannels);
  double cost;
  return ssc_best_split((T + kSscTile - 1) / kSscTile, units, ssc_resident(ssc_backward_bytes(es, NB), 2),
                        {0.3, 0.25, 0.05, 2.0 / NB, 0.5}, cost);
}

// Forward: parts of the tokens, and lanes that share two channels.  A block's 4 warps take 64 / lanes
// channels each.  (bf16, no kept states, us: 8 x 2048 x 2048 x 16, 128 blocks, one part 305, 4 287, 8 266;
// 12 x 1024 x 2048, 32 states, 384 blocks, one 373, 4 535; 4 x 1024 x 2048, 128 states, of which a block
// fills an SM, one 696, 8 1049, 16 1337.)  A tile takes 4 lanes 0.72 of the time that it takes 2, for half
// the channels; more than 16 states are always 4 lanes'.  Rows that are read value by value wait more than
// they compute, so that blocks hardly slow each other, and 4 lanes take 0.57 (bf16, 13 states, us:
// 1 x 2048 x 1023, one part, 2 lanes 958, 4 551; 8 x 2048 x 2047, 2 lanes in 8 parts 547, 4 in 2 500;
// 24 x 1024 x 2047, one part, 549 and 618).
struct SscForwardPlan {
  SscSplit split;
  int lanes;
};
inline SscForwardPlan ssc_forward_plan(long long B, long long T, long long D, long long N, long long G, int es, bool singles) {
  const long long tiles = (T + kSscTile - 1) / kSscTile;
  const int NB = (int)((N + 15) / 16);
  const SscCost c = singles ? SscCost{0.05, 0.7, 0.15, 2.0 / NB, 0} : SscCost{0.25, 0.8, 0.1, 2.0 / NB, 1.25};
  const auto blocks = [&](int lanes) {
    const long long width = 64 / lanes;
    return (B * G * ((D / G + width - 1) / width) + 3) / 4;
  };
  double cost, cost2;
  const SscForwardPlan four = {ssc_best_split(tiles, blocks(4), ssc_resident(ssc_forward_bytes(es, 4, NB), NB > 1 ? 3 : 4), c, cost), 4};
  if (NB > 1) return four;
  const SscForwardPlan two = {ssc_best_split(tiles, blocks(2), singles ? 3 : 4, c, cost2), 2};
  return (singles ? 0.57 : 0.72) * cost < cost2 ? four : two;
}
// Parts that scratch has to hold: of values of es bytes however the rows lie, or (es = 0) of any type.
inline long long ssc_most_parts(long long B, long long T, long long D, long long N, long long G, int es, bool backward) {
  if (es == 0) {
    const long long two = ssc_most_parts(B, T, D, N, G, 2, backward), four = ssc_most_parts(B, T, D, N, G, 4, backward);
    return two > four ? two : four;
  }
  if (backward) return ssc_backward_split(B, T, D, N, G, es).parts;
  const long long a = ssc_forward_plan(B, T, D, N, G, es, false).split.parts;
  const long long b = es == 2 ? ssc_forward_plan(B, T, D, N, G, es, true).split.parts : a;
  return a > b ? a : b;
}
inline size_t ssc_temp_bytes(long long B, long long T, long long D, long long N, long long G, int es, bool backward) {
  const long long parts = ssc_most_parts(B, T, D, N, G, es, backward);
  size_t floats = (size_t)B * (parts - 1) * (D * N + D + 1);
  if (backward) {
    floats += (size_t)B * parts * D * (N + 2);
    floats += 2 * (size_t)((D / G + kSscChannels - 1) / kSscChannels) * B * T * G * N;
  }
  return round_up(floats * sizeof(float), 256);
}

struct SelectiveScanStepJob {
  long long B = 0, D = 0, N = 0, G = 0, pool = 0;
  int softplus = 0;
  const void *x = nullptr, *dt = nullptr, *z = nullptr, *b = nullptr, *c = nullptr;
  long long sx = 0, sdt = 0, sz = 0, sy = 0, sb = 0, sbg = 0, sc = 0, scg = 0;  // row (and group) strides
  const float *a = nullptr, *d = nullptr, *bias = nullptr;
  float* state = nullptr;          // (pool, D, N)
  const int32_t* slots = nullptr;  // (B) or null
  void* y = nullptr;
};

constexpr int kVerifyMaxCluster = 8;

// Verification of up to K drafted tokens for each of B requests over a vocabulary of V.
struct VerifyJob {
  long long B = 0, K = 0, V = 0;
  const void* tokens = nullptr;    // (B, K) int32 or int64
  int tokens64 = 0;
  const void *target = nullptr, *draft = nullptr;  // (B, K + 1, V), (B, K, V) or null
  long long tb = 0, tt = 0, qb = 0, qt = 0;
  const float *accept = nullptr, *sample = nullptr;  // (B, K), (B)
  const int32_t* lengths = nullptr;                  // (B) or null: K
  int32_t *accepted = nullptr, *out = nullptr;       // (B), (B, K + 1)
};

template <class T> cudaError_t launch_causal_conv(const CausalConvJob& job, const LaunchCtx& ctx);
template <class T> cudaError_t launch_causal_conv_backward(const CausalConvJob& job, const LaunchCtx& ctx);
template <class T> cudaError_t launch_causal_conv_step(const CausalConvStepJob& job, const LaunchCtx& ctx);
template <class T> cudaError_t launch_selective_scan(const SelectiveScanJob& job, const LaunchCtx& ctx);
template <class T> cudaError_t launch_selective_scan_backward(const SelectiveScanJob& job, const LaunchCtx& ctx);
template <class T> cudaError_t launch_selective_scan_step(const SelectiveScanStepJob& job, const LaunchCtx& ctx);
template <class T> cudaError_t launch_verify(const VerifyJob& job, const LaunchCtx& ctx);

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
