// hnd_ffn_few.cuh -- the feed-forward block at a few positions (32 at most),
// as when a model is stepped token by token.
//
// What bounds it is reading the weights once: 2 operations a weight and
// position.  The tiles of hnd_ffn_gemm.cuh would hold 256 positions and leave
// most SMs without a tile, so here 16 rows of a weight make a block, its
// warps share the row's depth, and the positions are the narrow side of
// mma.sync (m16n8k16), which is far from a limit at this size.  Operands go
// from memory to registers without a stop: a thread loads 16 bytes, eight
// neighbouring k, of each of its rows, and since a sum over k may run in any
// order, the fragments' k are simply these (weights and positions alike).
// The warps' sums meet in shared memory.
//
// C 2048, F 5632, 4 positions, bf16 (69 MB of weights): 19.8 us a pass, 62 us
// with the large tiles.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "hnd_ffn_gemm.cuh"
#include "hnd_io.cuh"

namespace hnd {
namespace ffn {

constexpr int kFewMost = 32;

struct FewParams {
  const void *w0, *w1;         // [rows][K] in the activations' type; w1: the up projection
  const __nv_bfloat16* x;      // [plane][T][K]
  long long x_plane;
  int T, rows, K, act;
  __nv_bfloat16* hid;          // DUAL: [plane][T][rows]
  long long hid_plane;
  void* y;                     // else: element (row, t) at (t / L) rows L + row L + t % L
  int L;
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Eight neighbouring k of a row as packed bf16, plane by plane.
template <bool F32>
struct Eight {
  uint32_t v[F32 ? 3 : 1][4];
};
__device__ __forceinline__ uint4 stream16(const void* p) { return __ldcs(HND_G(reinterpret_cast<const uint4*>(p))); }

template <bool F32>
struct RawEight {
  uint4 u[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* w, long long at, bool there) {
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i)
      u[i] = there ? stream16(static_cast<const char*>(w) + (at + 4 * i) * (F32 ? 4 : 2)) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void planes(Eight<F32>& e) const {
    if constexpr (F32) {
      const uint32_t f[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        split3x2(__uint_as_float(f[2 * i]), __uint_as_float(f[2 * i + 1]), e.v[0][i], e.v[1][i], e.v[2][i]);
    } else {
      e.v[0][0] = u[0].x, e.v[0][1] = u[0].y, e.v[0][2] = u[0].z, e.v[0][3] = u[0].w;
    }
  }
};

// NT blocks of eight positions.  DUAL: H = act(w0 x) (w1 x), else y = w0 x.
template <bool F32, int NT, bool DUAL>
__global__ void __launch_bounds__(DUAL ? 256 : 512) k_ffn_few(const FewParams p) {
  constexpr int MATS = DUAL ? 2 : 1, U = F32 ? 2 : 4;      // chunks of 32 k in flight
  extern __shared__ __align__(16) unsigned char hnd_dyn_smem[];
  float* red = reinterpret_cast<float*>(hnd_dyn_smem);     // [warp][mat][position][row]
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
  const int row0 = blockIdx.x * 16, chunks = (p.K + 31) / 32;
  const long long ra = static_cast<long long>(min(row0 + g, p.rows - 1)) * p.K,
                  rb = static_cast<long long>(min(row0 + g + 8, p.rows - 1)) * p.K;
  const void* w[2] = {p.w0, p.w1};
  float acc[MATS][NT][4] = {};
  bool waited = false;
  for (int c0 = warp; c0 < chunks; c0 += U * warps) {
    RawEight<F32> raw[U][MATS][2];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int k = (c0 + i * warps) * 32 + q * 8;
#pragma unroll
      for (int m = 0; m < MATS; ++m) {
        raw[i][m][0].load(w[m], ra + k, k < p.K);
        raw[i][m][1].load(w[m], rb + k, k < p.K);
      }
    }
    if (!waited) {      // the weights are there before the kernel in front is done, its results are not
      asm volatile("griddepcontrol.wait;" ::: "memory");
      waited = true;
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int k = (c0 + i * warps) * 32 + q * 8;
      Eight<F32> a[MATS][2];
#pragma unroll
      for (int m = 0; m < MATS; ++m) raw[i][m][0].planes(a[m][0]), raw[i][m][1].planes(a[m][1]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int t = n * 8 + g;
        const bool there = t < p.T && k < p.K;
        uint4 b[F32 ? 3 : 1];
#pragma unroll
        for (int l = 0; l < (F32 ? 3 : 1); ++l)
          b[l] = there ? *HND_G(reinterpret_cast<const uint4*>(p.x + l * p.x_plane + static_cast<long long>(t) * p.K + k))
                       : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
          float part[4] = {};      // fp32: the tensor core truncates its sums, so they stay short
          float(&d)[4] = F32 ? part : acc[m][n];
#pragma unroll
          for (int cb = 0; cb < (F32 ? 6 : 1); ++cb) {
            int pa = 0, pb = 0;
            if (F32) planes_of(cb, pa, pb);
            const uint32_t lo[4] = {a[m][0].v[pa][0], a[m][1].v[pa][0], a[m][0].v[pa][1], a[m][1].v[pa][1]};
            const uint32_t hi[4] = {a[m][0].v[pa][2], a[m][1].v[pa][2], a[m][0].v[pa][3], a[m][1].v[pa][3]};
            mma16816(d, lo, b[pb].x, b[pb].y);
            mma16816(d, hi, b[pb].z, b[pb].w);
          }
          if (F32)
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[m][n][v] += part[v];
        }
      }
    }
  }
  if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
#pragma unroll
  for (int m = 0; m < MATS; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i)      // rows g and g + 8, positions 2 q and 2 q + 1
        *HND_S(red + ((warp * MATS + m) * NT * 8 + n * 8 + 2 * q + (i & 1)) * 16 + g + 8 * (i >> 1)) = acc[m][n][i];
  __syncthreads();
  for (int i = threadIdx.x; i < NT * 128; i += blockDim.x) {
    const int t = i / 16, row = row0 + i % 16;
    if (t >= p.T || row >= p.rows) continue;
    float s[MATS];
#pragma unroll
    for (int m = 0; m < MATS; ++m) {
      s[m] = 0.f;
      for (int v = 0; v < warps; ++v) s[m] += *HND_S(red + (v * MATS + m) * NT * 128 + i);
    }
    if constexpr (DUAL) {
      const float gv[2] = {s[0], s[0]}, uv[2] = {s[1], s[1]};
      float h[2];
      if (p.act)
        hidden2<true, 1>(gv, uv, h);
      else
        hidden2<true, 0>(gv, uv, h);
      __nv_bfloat16* o = p.hid + static_cast<long long>(t) * p.rows + row;
      if constexpr (F32) {
        __nv_bfloat16 v[3];
        split3(h[0], v[0], v[1], v[2]);
#pragma unroll
        for (int l = 0; l < 3; ++l) *HND_G(o + l * p.hid_plane) = v[l];
      } else {
        *HND_G(o) = __float2bfloat16_rn(h[0]);
      }
    } else {
      const long long at = static_cast<long long>(t / p.L) * p.rows * p.L + static_cast<long long>(row) * p.L + t % p.L;
      if constexpr (F32)
        st1(static_cast<float*>(p.y) + at, s[0]);
      else
        st1(static_cast<__nv_bfloat16*>(p.y) + at, s[0]);
    }
  }
}

}  // namespace ffn
}  // namespace hnd
