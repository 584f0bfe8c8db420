// Counter-based dropout over a flat tensor.
#include "hnd_block.h"
#include "hnd_io.cuh"
#include "hnd_philox.cuh"

namespace hnd {

template <class T>
__global__ void __launch_bounds__(256) k_dropout(const T* __restrict__ x, T* __restrict__ y, long long count,
                                                 unsigned border, float factor, const int64_t* __restrict__ rng) {
  const DropState s = border ? drop_state(rng) : DropState{};
  const long long groups = (count + 7) / 8;
  for (long long g = blockIdx.x * 256LL + threadIdx.x; g < groups; g += gridDim.x * 256LL) {
    const uint4 w = border ? drop_lots(s, static_cast<uint64_t>(g)) : make_uint4(0, 0, 0, 0);
    for (int j = 0; j < 8 && 8 * g + j < count; ++j) {
      const float v = ld1(x + 8 * g + j);
      st1(y + 8 * g + j, drop_lot(w, j) >= border ? v * factor : 0.f);
    }
  }
}

cudaError_t launch_dropout(long long count, int bf16, const DropStage& d, const void* x, void* y, cudaStream_t st) {
  long long blocks = ((count + 7) / 8 + 255) / 256;
  if (blocks > 148 * 8) blocks = 148 * 8;
  if (bf16)
    k_dropout<<<static_cast<unsigned>(blocks), 256, 0, st>>>(static_cast<const __nv_bfloat16*>(x),
                                                             static_cast<__nv_bfloat16*>(y), count, d.border,
                                                             d.factor, d.rng);
  else
    k_dropout<<<static_cast<unsigned>(blocks), 256, 0, st>>>(static_cast<const float*>(x), static_cast<float*>(y),
                                                             count, d.border, d.factor, d.rng);
  return cudaGetLastError();
}

}  // namespace hnd
