// abi.h -- what the entry points share: the launch settings of a call, the record of a
// failed CUDA call, caller-supplied or stream-ordered scratch.  Defined in api.cu.
#pragma once

#include "launch.h"

namespace gbs {

int abi_ctx(void* stream, LaunchCtx& ctx);  // GB_OK, GB_ERR_CUDA or GB_ERR_UNSUPPORTED
int abi_cuda_fail(cudaError_t e);           // remembers e, returns GB_ERR_CUDA

// Scratch of one call; what the library allocated is freed when the call ends.
struct Temp {
  void* p = nullptr;
  bool owned = false;
  cudaStream_t s = nullptr;
  ~Temp() {
    if (owned && p) cudaFreeAsync(p, s);
  }
};
int abi_temp(void* temp, size_t temp_bytes, size_t need, cudaStream_t s, Temp& t);

}  // namespace gbs
