// hnd_block.h -- host-side launchers of the operators around the convolution
// (hnd_block_api.cu checks the arguments and calls them).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace hnd {

// One norm stage: kind as hyena_nd_norm_kind (0 none, 1 RMS, 2 layer).
struct NormStage {
  int kind = 0;
  float eps = 0.f;
  const float* w = nullptr;
  const float* b = nullptr;
};

// Dropout: lots below `border` (of 65536) are dropped, the rest multiplied by
// `factor`; border 0 = no dropout.
struct DropStage {
  unsigned border = 0;
  float factor = 1.f;
  const int64_t* rng = nullptr;
};

struct JoinArgs {
  long long B = 0, C = 0, L = 0;
  int bf16 = 0;
  NormStage post, pre;
  const float *gate = nullptr, *scale = nullptr;
  DropStage drop;
  const void *x = nullptr, *y = nullptr;      // y null: the norm alone (h = x, not written)
  void *h = nullptr, *n = nullptr;
  const void *dh = nullptr, *dn = nullptr;    // either may be null (zero)
  void *dx = nullptr, *dy = nullptr;
  float *dpost_w = nullptr, *dpost_b = nullptr, *dgate = nullptr, *dscale = nullptr, *dpre_w = nullptr,
        *dpre_b = nullptr;
  void* ws = nullptr;
  cudaStream_t stream = nullptr;
};

// bounds_register for these operators: a call without a status word of its own
// records in the library's, which hyena_nd_device_status reads for a null
// workspace.
struct BoundsList;
cudaError_t register_buffers(const BoundsList& list, int* status, cudaStream_t st);

cudaError_t launch_join_forward(const JoinArgs& a);
cudaError_t launch_join_backward(const JoinArgs& a);
size_t join_workspace(long long B, long long C, long long L, int bf16);

cudaError_t launch_dropout(long long count, int bf16, const DropStage& d, const void* x, void* y, cudaStream_t st);

struct FfnArgs {
  long long B = 0, C = 0, L = 0, F = 0;
  int bf16 = 0, act = 0;
  const void *x = nullptr, *wg = nullptr, *wu = nullptr, *wd = nullptr, *dy = nullptr;
  void *y = nullptr, *dx = nullptr, *dwg = nullptr, *dwu = nullptr, *dwd = nullptr;
  int* status = nullptr;
  void* ws = nullptr;
  cudaStream_t stream = nullptr;
};

cudaError_t launch_ffn_forward(const FfnArgs& a);
cudaError_t launch_ffn_backward(const FfnArgs& a);
size_t ffn_workspace(const FfnArgs& a, bool backward);

}  // namespace hnd
