// Counter-based dropout over a flat tensor: y_i = m_i x_i, the mask bits from
// Philox4x32-10 at (seed, offset, i / 8).
//
// Bound by memory (two bytes moved a byte of activations) as long as the ten
// rounds, some 60 integer operations for eight elements, stay hidden behind
// it: a thread takes eight elements, one counter, as one or two 16-byte
// loads, four groups in flight.  32 x 128^3 bf16: 53 us, 77% of the rate of a
// copy.
#include "hnd_block.h"
#include "hnd_io.cuh"
#include "hnd_philox.cuh"

namespace hnd {

// The eight elements of a group as 16-byte words: bf16 one, fp32 two.
template <class TT>
struct Group8 {
  static constexpr int W = sizeof(TT) / 2;
  uint4 u[W];
};

__device__ __forceinline__ void drop8(Group8<__nv_bfloat16>& g, const uint4& lots, uint32_t border, float factor) {
  const uint32_t l[4] = {lots.x, lots.y, lots.z, lots.w};
  uint32_t* w = &g.u[0].x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = __uint_as_float(w[i] << 16) * factor, b = __uint_as_float(w[i] & 0xFFFF0000u) * factor;
    const __nv_bfloat162 h = __floats2bfloat162_rn((l[i] & 0xFFFFu) >= border ? a : 0.f, (l[i] >> 16) >= border ? b : 0.f);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
}
__device__ __forceinline__ void drop8(Group8<float>& g, const uint4& lots, uint32_t border, float factor) {
  const uint32_t l[4] = {lots.x, lots.y, lots.z, lots.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t* w = i < 2 ? &g.u[0].x : &g.u[1].x;
    uint32_t &a = w[2 * (i & 1)], &b = w[2 * (i & 1) + 1];
    a = (l[i] & 0xFFFFu) >= border ? __float_as_uint(__uint_as_float(a) * factor) : 0u;
    b = (l[i] >> 16) >= border ? __float_as_uint(__uint_as_float(b) * factor) : 0u;
  }
}

constexpr int kThreads = 256, kFlight = 4;

template <class TT>
__global__ void __launch_bounds__(kThreads) k_dropout(const TT* __restrict__ x, TT* __restrict__ y, long long count,
                                                      unsigned border, float factor,
                                                      const int64_t* __restrict__ rng) {
  constexpr int W = Group8<TT>::W;
  const DropState s = border ? drop_state(rng) : DropState{};
  const long long whole = count / 8;
  const uint4* in = reinterpret_cast<const uint4*>(x);
  uint4* out = reinterpret_cast<uint4*>(y);
  for (long long g0 = blockIdx.x * static_cast<long long>(kThreads * kFlight) + threadIdx.x; g0 < whole;
       g0 += gridDim.x * static_cast<long long>(kThreads * kFlight)) {
    Group8<TT> v[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f)
      if (g0 + f * kThreads < whole)
#pragma unroll
        for (int q = 0; q < W; ++q) v[f].u[q] = __ldcs(HND_G(in + (g0 + f * kThreads) * W + q));
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const long long g = g0 + f * kThreads;
      if (g >= whole) continue;
      if (border) drop8(v[f], drop_lots(s, static_cast<uint64_t>(g)), border, factor);
#pragma unroll
      for (int q = 0; q < W; ++q) __stcs(HND_G(out + g * W + q), v[f].u[q]);
    }
  }
  // the last, shorter group
  const int rest = static_cast<int>(count - 8 * whole);
  if (blockIdx.x == 0 && threadIdx.x < rest) {
    const long long i = 8 * whole + threadIdx.x;
    const float v = ld1(x + i);
    const uint32_t lot = border ? drop_lot(drop_lots(s, static_cast<uint64_t>(whole)), threadIdx.x) : 0u;
    st1(y + i, lot >= border ? v * factor : 0.f);
  }
}

template <class TT>
static cudaError_t run(long long count, const DropStage& d, const void* x, void* y, cudaStream_t st) {
  long long blocks = (count / 8 + kThreads * kFlight - 1) / (kThreads * kFlight);
  if (blocks < 1) blocks = 1;
  if (blocks >= 1LL << 31) blocks = (1LL << 31) - 1;
  k_dropout<TT><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(static_cast<const TT*>(x), static_cast<TT*>(y), count,
                                                                    d.border, d.factor, d.rng);
  return cudaGetLastError();
}

cudaError_t launch_dropout(long long count, int bf16, const DropStage& d, const void* x, void* y, cudaStream_t st) {
  return bf16 ? run<__nv_bfloat16>(count, d, x, y, st) : run<float>(count, d, x, y, st);
}

}  // namespace hnd
