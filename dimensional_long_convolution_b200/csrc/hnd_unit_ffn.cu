// The gated feed-forward block over the channels of each position.
#include "hnd_block.h"
#include "hnd_io.cuh"

namespace hnd {

// A matrix whose column j lies at (j / L) bs + j % L and whose row i adds i rs:
// activations [B, C, L] are such a matrix [C, B L], weights one with L = cols.
template <class TT>
struct View {
  TT* p;
  long long L, bs, rs;
  __device__ TT* at(long long i, long long j) const { return p + (j / L) * bs + i * rs + j % L; }
};

__device__ __forceinline__ float act_value(int act, float g) {
  return act ? g * 0.5f * (1.f + erff(g * 0.70710678118654752f)) : g / (1.f + expf(-g));
}
__device__ __forceinline__ float act_slope(int act, float g) {
  if (act) return 0.5f * (1.f + erff(g * 0.70710678118654752f)) + g * 0.39894228040143268f * expf(-0.5f * g * g);
  const float s = 1.f / (1.f + expf(-g));
  return s * (1.f + g * (1.f - s));
}

constexpr int kGT = 64, kGK = 16;

// acc += A B over k, A(m, k) = a(m, k) or a(k, m) (TA), B(k, n) = b(k, n) or b(n, k) (TB).
template <bool TA, bool TB, class TT>
__device__ __forceinline__ void tile_product(float (&acc)[4][4], const View<const TT>& a, const View<const TT>& b,
                                             long long M, long long N, long long K, long long m0, long long n0,
                                             float (*sa)[kGT + 1], float (*sb)[kGT + 1]) {
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  float part[4][4] = {};      // sums of 256 terms at a time keep the rounding of long sums small
  for (long long k0 = 0; k0 < K; k0 += kGK) {
    __syncthreads();
    for (int i = tid; i < kGT * kGK; i += 256) {
      const int k = TA ? i / kGT : i % kGK, m = TA ? i % kGT : i / kGK;
      sa[k][m] = (m0 + m < M && k0 + k < K) ? ld1(TA ? a.at(k0 + k, m0 + m) : a.at(m0 + m, k0 + k)) : 0.f;
    }
    for (int i = tid; i < kGT * kGK; i += 256) {
      const int k = TB ? i % kGK : i / kGT, n = TB ? i / kGK : i % kGT;
      sb[k][n] = (n0 + n < N && k0 + k < K) ? ld1(TB ? b.at(n0 + n, k0 + k) : b.at(k0 + k, n0 + n)) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kGK; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) part[i][q] += sa[k][ty * 4 + i] * sb[k][tx * 4 + q];
    if (k0 % 256 == 256 - kGK || k0 + kGK >= K)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][q] += part[i][q], part[i][q] = 0.f;
  }
}

#define FFN_TILE                                                              \
  __shared__ float sa[kGK][kGT + 1], sb[kGK][kGT + 1];                        \
  const long long m0 = blockIdx.y * static_cast<long long>(kGT), n0 = blockIdx.x * static_cast<long long>(kGT); \
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;

// H = act(Wg X) (Wu X)
template <class TT>
__global__ void __launch_bounds__(256) k_ffn_hidden(View<const TT> x, View<const TT> wg, View<const TT> wu,
                                                    View<TT> h, long long C, long long F, long long T, int act) {
  FFN_TILE
  float g[4][4] = {}, u[4][4] = {};
  tile_product<false, false>(g, wg, x, F, T, C, m0, n0, sa, sb);
  tile_product<false, false>(u, wu, x, F, T, C, m0, n0, sa, sb);
  for (int i = 0; i < 4; ++i)
    for (int q = 0; q < 4; ++q) {
      const long long m = m0 + ty * 4 + i, n = n0 + tx * 4 + q;
      if (m < F && n < T) st1(h.at(m, n), act_value(act, g[i][q]) * u[i][q]);
    }
}

// H, dG, dU from X and dY
template <class TT>
__global__ void __launch_bounds__(256)
    k_ffn_hidden_grad(View<const TT> x, View<const TT> dy, View<const TT> wg, View<const TT> wu, View<const TT> wd,
                      View<TT> h, View<TT> dg, View<TT> du, long long C, long long F, long long T, int act) {
  FFN_TILE
  float g[4][4] = {}, u[4][4] = {}, d[4][4] = {};
  tile_product<false, false>(g, wg, x, F, T, C, m0, n0, sa, sb);
  tile_product<false, false>(u, wu, x, F, T, C, m0, n0, sa, sb);
  tile_product<true, false>(d, wd, dy, F, T, C, m0, n0, sa, sb);
  for (int i = 0; i < 4; ++i)
    for (int q = 0; q < 4; ++q) {
      const long long m = m0 + ty * 4 + i, n = n0 + tx * 4 + q;
      if (m >= F || n >= T) continue;
      const float a = act_value(act, g[i][q]);
      st1(h.at(m, n), a * u[i][q]);
      st1(dg.at(m, n), d[i][q] * u[i][q] * act_slope(act, g[i][q]));
      st1(du.at(m, n), d[i][q] * a);
    }
}

// D = A1 B1 (+ A2 B2)
template <bool TA, bool TB, class TT>
__global__ void __launch_bounds__(256)
    k_ffn_product(View<const TT> a1, View<const TT> b1, View<const TT> a2, View<const TT> b2, View<TT> d, long long M,
                  long long N, long long K) {
  FFN_TILE
  float acc[4][4] = {};
  tile_product<TA, TB>(acc, a1, b1, M, N, K, m0, n0, sa, sb);
  if (a2.p) tile_product<TA, TB>(acc, a2, b2, M, N, K, m0, n0, sa, sb);
  for (int i = 0; i < 4; ++i)
    for (int q = 0; q < 4; ++q) {
      const long long m = m0 + ty * 4 + i, n = n0 + tx * 4 + q;
      if (m < M && n < N) st1(d.at(m, n), acc[i][q]);
    }
}

static dim3 tiles(long long M, long long N) {
  return dim3(static_cast<unsigned>((N + kGT - 1) / kGT), static_cast<unsigned>((M + kGT - 1) / kGT));
}

template <class TT>
struct Ffn {
  const FfnArgs& a;
  long long T = a.B * a.L;
  template <class Q>
  View<Q> grid(Q* p) const {
    return {p, a.L, a.C * a.L, a.L};
  }
  template <class Q>
  View<Q> flat(Q* p, long long cols) const {
    return {p, cols, 0, cols};
  }
  const TT* in(const void* p) const { return static_cast<const TT*>(p); }
  TT* out(void* p) const { return static_cast<TT*>(p); }
  TT* hidden(int i) const { return out(a.ws) + static_cast<size_t>(i) * T * a.F; }

  cudaError_t forward() const {
    k_ffn_hidden<TT><<<tiles(a.F, T), 256, 0, a.stream>>>(grid(in(a.x)), flat(in(a.wg), a.C), flat(in(a.wu), a.C),
                                                          flat(hidden(0), T), a.C, a.F, T, a.act);
    k_ffn_product<false, false, TT><<<tiles(a.C, T), 256, 0, a.stream>>>(
        flat(in(a.wd), a.F), flat(in(hidden(0)), T), View<const TT>{}, View<const TT>{}, grid(out(a.y)), a.C, T, a.F);
    return cudaGetLastError();
  }
  cudaError_t backward() const {
    const auto x = grid(in(a.x)), dy = grid(in(a.dy));
    const auto wg = flat(in(a.wg), a.C), wu = flat(in(a.wu), a.C);
    const auto h = flat(in(hidden(0)), T), dg = flat(in(hidden(1)), T), du = flat(in(hidden(2)), T);
    const View<const TT> none{};
    k_ffn_hidden_grad<TT><<<tiles(a.F, T), 256, 0, a.stream>>>(x, dy, wg, wu, flat(in(a.wd), a.F), flat(hidden(0), T),
                                                               flat(hidden(1), T), flat(hidden(2), T), a.C, a.F, T,
                                                               a.act);
    k_ffn_product<true, false, TT><<<tiles(a.C, T), 256, 0, a.stream>>>(wg, dg, wu, du, grid(out(a.dx)), a.C, T, a.F);
    k_ffn_product<false, true, TT>
        <<<tiles(a.F, a.C), 256, 0, a.stream>>>(dg, x, none, none, flat(out(a.dwg), a.C), a.F, a.C, T);
    k_ffn_product<false, true, TT>
        <<<tiles(a.F, a.C), 256, 0, a.stream>>>(du, x, none, none, flat(out(a.dwu), a.C), a.F, a.C, T);
    k_ffn_product<false, true, TT>
        <<<tiles(a.C, a.F), 256, 0, a.stream>>>(dy, h, none, none, flat(out(a.dwd), a.F), a.C, a.F, T);
    return cudaGetLastError();
  }
};

size_t ffn_workspace(const FfnArgs& a, bool backward) {
  return static_cast<size_t>(backward ? 3 : 1) * a.B * a.L * a.F * (a.bf16 ? 2 : 4);
}

cudaError_t launch_ffn_forward(const FfnArgs& a) {
  return a.bf16 ? Ffn<__nv_bfloat16>{a}.forward() : Ffn<float>{a}.forward();
}

cudaError_t launch_ffn_backward(const FfnArgs& a) {
  return a.bf16 ? Ffn<__nv_bfloat16>{a}.backward() : Ffn<float>{a}.backward();
}

}  // namespace hnd
