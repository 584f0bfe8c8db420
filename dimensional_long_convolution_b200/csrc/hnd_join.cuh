// hnd_join.cuh -- the residual join in one pass over memory.
//
// h = x + scale gate m norm_post(y), n = norm_pre(h) and their gradients are
// bound by memory: each activation should cross it once.  So a block keeps
// all channels of a few positions in registers, from the loads through the
// statistics to the stores, and a mean or a sum over the channels is a
// reduction between the block's threads: within warps by shuffles, between
// them through shared memory.  Variances are taken around the mean in a second
// sweep over the registers, which costs no memory and loses nothing where the
// mean is far from zero.
//
// Grid layout [B, C, L]: W neighbouring lanes hold V neighbouring positions
// each (16 bytes), the rest of the block's threads the channels, K apiece.  W
// is as wide as the registers allow: 8 lanes make 128-byte rows, and 4, 2 or 1
// lanes hold more channels.  Token layout (L = 1): the channels of a position
// lie together, V to a thread and K such vectors, and a group of threads holds
// a position.  Rows that are no multiple of 16 bytes take V = 1.
#pragma once

#include "hnd_block.h"
#include "hnd_io.cuh"
#include "hnd_philox.cuh"

namespace hnd {

// Everything a kernel needs of a join, by value.
struct JoinDev {
  long long B, C, L, T;
  int post, pre;
  float eps1, eps2;
  const float *w1, *b1, *w2, *b2, *gate, *scale;
  unsigned border;
  float factor;
  const int64_t* rng;
};

// The persistent kernels of hnd_join_grid.cuh: K channels of a thread, w
// lanes of positions, and (gradients) `chunks` blocks a sample.
cudaError_t launch_join_grid_fwd(const JoinArgs& a, const JoinDev& j, int w, int K, unsigned blocks);
cudaError_t launch_join_grid_bwd(const JoinArgs& a, const JoinDev& j, int w, int K, int chunks, unsigned blocks,
                                 float4* part);

// V neighbouring values as they are stored.
template <class TT, int V>
struct alignas(sizeof(TT) * V) Raw {
  TT v[V];
};
template <int V>
__device__ __forceinline__ float raw_at(const Raw<float, V>& r, int i) {
  return r.v[i];
}
template <int V>
__device__ __forceinline__ float raw_at(const Raw<__nv_bfloat16, V>& r, int i) {
  return __bfloat162float(r.v[i]);
}
template <class TT, int V>
__device__ __forceinline__ Raw<TT, V> raw_load(const TT* p) {
  if constexpr (sizeof(TT) * V == 16) {
    const uint4 u = __ldcs(HND_G(reinterpret_cast<const uint4*>(p)));
    return *reinterpret_cast<const Raw<TT, V>*>(&u);
  } else {
    return *HND_G((reinterpret_cast<const Raw<TT, V>*>(p)));
  }
}
__device__ __forceinline__ void raw_set(float& d, float v) { d = v; }
__device__ __forceinline__ void raw_set(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }
template <class TT, int V>
__device__ __forceinline__ void raw_store(TT* p, const float (&f)[V]) {
  Raw<TT, V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) raw_set(r.v[i], f[i]);
  if constexpr (sizeof(TT) * V == 16)
    __stcs(HND_G(reinterpret_cast<uint4*>(p)), *reinterpret_cast<const uint4*>(&r));
  else
    *HND_G((reinterpret_cast<Raw<TT, V>*>(p))) = r;
}

// Bit v: element i0 + v stays.  i0 is a multiple of V.
template <int V>
__device__ __forceinline__ unsigned keep_bits(const DropState& ds, unsigned border, long long i0) {
  const uint4 w = drop_lots(ds, static_cast<uint64_t>(i0 >> 3));
  unsigned bits = 0;
  if constexpr (V == 1) {
    bits = drop_lot(w, static_cast<int>(i0 & 7)) >= border;
  } else {
    const bool upper = V == 4 && (i0 & 4);
    const uint32_t u[4] = {upper ? w.z : w.x, upper ? w.w : w.y, w.z, w.w};
#pragma unroll
    for (int v = 0; v < V; ++v) bits |= static_cast<unsigned>(((v & 1) ? u[v / 2] >> 16 : u[v / 2] & 0xFFFFu) >= border) << v;
  }
  return bits;
}

constexpr int kJoinMaxThreads = 512;

// Where a thread's values lie.  TOK: K vectors of V channels of one position;
// else K channels of V positions.
template <class TT, int V, int K, bool TOK>
struct Tile {
  static constexpr int P = TOK ? 1 : V;     // positions of a thread
  const JoinDev& j;
  int lanes;              // grid: W; token: threads of a position
  int lane, cg, groups;   // grid: lane of W, channel row, rows; token: thread of the position, 0, positions a block
  int flip = 0;
  float* buf;             // [2][warps][lanes of a warp that hold sums][values]
  long long base = 0, b = 0;
  bool live = false;

  __device__ Tile(const JoinDev& jj, int w, float* smem) : j(jj), lanes(w), buf(smem) {
    lane = threadIdx.x % w;
    cg = threadIdx.x / w;
    groups = blockDim.x / w;
  }
  __device__ static constexpr int slot(int v) { return TOK ? 0 : v; }
  __device__ long long chan(int k) const {      // the channel of vector k (its first)
    return TOK ? (static_cast<long long>(lane) + static_cast<long long>(k) * lanes) * V
               : cg + static_cast<long long>(k) * groups;
  }
  __device__ bool has(int k) const { return live && chan(k) < j.C; }
  __device__ long long at(int k) const { return TOK ? base + chan(k) : base + chan(k) * j.L; }

  // Grid: unit u of V positions, units counted through the samples.
  __device__ void place(long long sample, long long l, bool ok) {
    live = ok;
    b = ok ? sample : 0;
    base = b * j.C * j.L + (ok ? l : 0);
  }
  // Sums over the channels of each of the thread's positions, N values each.
  template <int N>
  __device__ void sum(float (&s)[N][P]) {
    const int warps = blockDim.x / 32, warp = threadIdx.x / 32;
    const int first = TOK ? 1 : lanes;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int i = 0; i < P; ++i)
        for (int o = 16; o >= first; o >>= 1) s[n][i] += __shfl_xor_sync(0xFFFFFFFFu, s[n][i], o);
    if (TOK && lanes == 32) return;
    // what a warp writes: token: one set; grid: one of each of its (at most
    // 32) lanes, lanes side by side
    const int l = TOK ? 0 : lane, sets = TOK ? 1 : lanes;
    float* out = buf + (flip * warps + warp) * sets * (2 * P) + l;
    if ((threadIdx.x & 31) < sets)
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < P; ++i) *HND_S(out + (n * P + i) * sets) = s[n][i];
    __syncthreads();
    const int from = TOK ? warp / (lanes / 32) * (lanes / 32) : 0, to = TOK ? from + lanes / 32 : warps;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int i = 0; i < P; ++i) s[n][i] = 0.f;
    for (int w = from; w < to; ++w) {
      const float* in = buf + (flip * warps + w) * sets * (2 * P) + l;
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < P; ++i) s[n][i] += *HND_S(in + (n * P + i) * sets);
    }
    flip ^= 1;      // the next sums go to the other half: no second barrier
  }
  // Mean and reciprocal deviation of f(k, v) at each position.
  template <class Fn>
  __device__ void stats(int kind, float eps, float (&mu)[P], float (&rho)[P], Fn f) {
#pragma unroll
    for (int i = 0; i < P; ++i) mu[i] = 0.f, rho[i] = 1.f;
    if (!kind) return;
    const float inv = 1.f / static_cast<float>(j.C);
    float s[1][P];
    if (kind == 2) {
#pragma unroll
      for (int i = 0; i < P; ++i) s[0][i] = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (has(k))
#pragma unroll
          for (int v = 0; v < V; ++v) s[0][slot(v)] += f(k, v);
      sum(s);
#pragma unroll
      for (int i = 0; i < P; ++i) mu[i] = s[0][i] * inv;
    }
#pragma unroll
    for (int i = 0; i < P; ++i) s[0][i] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (has(k))
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float d = f(k, v) - mu[slot(v)];
          s[0][slot(v)] += d * d;
        }
    sum(s);
#pragma unroll
    for (int i = 0; i < P; ++i) rho[i] = rsqrtf(s[0][i] * inv + eps);
  }
  // A parameter of each channel: the same for a grid vector, V of them token-major.
  __device__ void param(const float* p, int k, float none, float (&o)[TOK ? V : 1]) const {
#pragma unroll
    for (int v = 0; v < (TOK ? V : 1); ++v) o[v] = p ? __ldg(HND_G(p + chan(k) + v)) : none;
  }
  // scale gate
  __device__ void both(int k, float (&o)[TOK ? V : 1]) const {
    param(j.scale, k, 1.f, o);
    if (j.gate)
#pragma unroll
      for (int v = 0; v < (TOK ? V : 1); ++v) o[v] *= __ldg(HND_G(j.gate + b * j.C + chan(k) + v));
  }
};
#define HND_PV(v) (TOK ? (v) : 0)      // index of a parameter of vector element v

// y's statistics and h: keep[k] has a bit per value.
template <class TT, int V, int K, bool TOK>
__device__ __forceinline__ void join_head(Tile<TT, V, K, TOK>& t, const TT* x, const TT* y, Raw<TT, V> (&ry)[K],
                                          unsigned (&keep)[K], float (&hv)[K][V],
                                          float (&mu1)[Tile<TT, V, K, TOK>::P], float (&rho1)[Tile<TT, V, K, TOK>::P]) {
  using TL = Tile<TT, V, K, TOK>;
  const JoinDev& j = t.j;
  Raw<TT, V> rx[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (t.has(k)) {
      if (y) ry[k] = raw_load<TT, V>(y + t.at(k));
      rx[k] = raw_load<TT, V>(x + t.at(k));
    }
    keep[k] = ~0u;
  }
  if (!y) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int v = 0; v < V; ++v) hv[k][v] = t.has(k) ? raw_at(rx[k], v) : 0.f;
    return;
  }
  if (j.border) {
    const DropState ds = drop_state(j.rng);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (t.has(k)) keep[k] = keep_bits<V>(ds, j.border, t.at(k));
  }
  t.stats(j.post, j.eps1, mu1, rho1, [&](int k, int v) { return raw_at(ry[k], v); });
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (!t.has(k)) {
#pragma unroll
      for (int v = 0; v < V; ++v) hv[k][v] = 0.f;
      continue;
    }
    float w[TOK ? V : 1], b[TOK ? V : 1], sg[TOK ? V : 1];
    t.param(j.w1, k, 1.f, w);
    t.param(j.b1, k, 0.f, b);
    t.both(k, sg);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float z = (raw_at(ry[k], v) - mu1[TL::slot(v)]) * rho1[TL::slot(v)] * w[HND_PV(v)] + b[HND_PV(v)];
      const float xv = raw_at(rx[k], v);
      hv[k][v] = (keep[k] >> v & 1u) ? xv + sg[HND_PV(v)] * (j.factor * z) : xv;
    }
  }
}

template <class TT, int V, int K, bool TOK>
__global__ void __launch_bounds__(kJoinMaxThreads)
    k_join_fwd(const JoinDev j, int w, const TT* __restrict__ x, const TT* __restrict__ y, TT* __restrict__ h,
               TT* __restrict__ n) {
  extern __shared__ __align__(16) unsigned char hnd_dyn_smem[];
  using TL = Tile<TT, V, K, TOK>;
  TL t(j, w, reinterpret_cast<float*>(hnd_dyn_smem));
  if (TOK) {
    const long long row = blockIdx.x * static_cast<long long>(t.groups) + t.cg;
    t.place(row, 0, row < j.B);
  } else {
    const long long per = j.L / V, u = blockIdx.x * static_cast<long long>(w) + t.lane, b = u / per;
    t.place(b, (u - b * per) * V, b < j.B);
  }
  Raw<TT, V> ry[K];
  unsigned keep[K];
  float hv[K][V], mu[TL::P], rho[TL::P];
  join_head<TT, V, K, TOK>(t, x, y, ry, keep, hv, mu, rho);
  if (h)
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (t.has(k)) raw_store<TT, V>(h + t.at(k), hv[k]);
  if (!n) return;
  t.stats(j.pre, j.eps2, mu, rho, [&](int k, int v) { return hv[k][v]; });
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (!t.has(k)) continue;
    float w2[TOK ? V : 1], b2[TOK ? V : 1];
    t.param(j.w2, k, 1.f, w2);
    t.param(j.b2, k, 0.f, b2);
#pragma unroll
    for (int v = 0; v < V; ++v)
      hv[k][v] = (hv[k][v] - mu[TL::slot(v)]) * rho[TL::slot(v)] * w2[HND_PV(v)] + b2[HND_PV(v)];
    raw_store<TT, V>(n + t.at(k), hv[k]);
  }
}

// Gradients.  A block goes through `tiles` of its sample (grid: chunk of
// `chunks` blocks a sample; token: all positions) and keeps each channel's
// sums of dht m yhat, dht m, dn hhat and dn over its positions, which it
// leaves in part[block or group][C]; token-major they are weighted with the
// gate, since every position has its own.
template <class TT, int V, int K, bool TOK>
__global__ void __launch_bounds__(kJoinMaxThreads)
    k_join_bwd(const JoinDev j, int w, int chunks, const TT* __restrict__ x, const TT* __restrict__ y,
               const TT* __restrict__ dh, const TT* __restrict__ dn, TT* __restrict__ dx, TT* __restrict__ dy,
               float* __restrict__ dgate, float4* __restrict__ part) {
  extern __shared__ __align__(16) unsigned char hnd_dyn_smem[];
  using TL = Tile<TT, V, K, TOK>;
  constexpr int A = TOK ? V : 1;      // channels of a vector that have sums of their own
  TL t(j, w, reinterpret_cast<float*>(hnd_dyn_smem));
  const float inv = 1.f / static_cast<float>(j.C);
  float4 acc[K][A];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int a = 0; a < A; ++a) acc[k][a] = make_float4(0.f, 0.f, 0.f, 0.f);
  const long long per = TOK ? 0 : j.L / V;
  const long long tiles = TOK ? (j.B + t.groups - 1) / t.groups : (per + w - 1) / w;
  const long long sample = TOK ? 0 : blockIdx.x / chunks;
  for (long long i = TOK ? blockIdx.x : blockIdx.x % chunks; i < tiles; i += TOK ? gridDim.x : chunks) {
    if (TOK) {
      const long long row = i * t.groups + t.cg;
      t.place(row, 0, row < j.B);
    } else {
      const long long u = i * w + t.lane;
      t.place(sample, u * V, u < per);
    }
    Raw<TT, V> ry[K], rdn[K], rdh[K];
    unsigned keep[K];
    float hv[K][V], mu1[TL::P], rho1[TL::P], mu2[TL::P], rho2[TL::P];
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (t.has(k)) {
        if (dn) rdn[k] = raw_load<TT, V>(dn + t.at(k));
        if (dh) rdh[k] = raw_load<TT, V>(dh + t.at(k));
      }
    join_head<TT, V, K, TOK>(t, x, y, ry, keep, hv, mu1, rho1);
    if (dn) {
      t.stats(j.pre, j.eps2, mu2, rho2, [&](int k, int v) { return hv[k][v]; });
      float s[2][TL::P];
#pragma unroll
      for (int q = 0; q < TL::P; ++q) s[0][q] = s[1][q] = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!t.has(k)) continue;
        float w2[A];
        t.param(j.w2, k, 1.f, w2);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float d = raw_at(rdn[k], v), a = d * w2[HND_PV(v)];
          hv[k][v] = (hv[k][v] - mu2[TL::slot(v)]) * rho2[TL::slot(v)];      // hhat from here on
          s[0][TL::slot(v)] += a;
          s[1][TL::slot(v)] += a * hv[k][v];
          acc[k][HND_PV(v)].z += d * hv[k][v];
          acc[k][HND_PV(v)].w += d;
        }
      }
      t.template sum<2>(s);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!t.has(k)) continue;
        float w2[A];
        t.param(j.w2, k, 1.f, w2);
#pragma unroll
        for (int v = 0; v < V; ++v) {      // dht from here on
          const int q = TL::slot(v);
          const float a = raw_at(rdn[k], v) * w2[HND_PV(v)];
          hv[k][v] = (dh ? raw_at(rdh[k], v) : 0.f) +
                     rho2[q] * (a - (j.pre == 2 ? s[0][q] * inv : 0.f) - hv[k][v] * (s[1][q] * inv));
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) hv[k][v] = dh && t.has(k) ? raw_at(rdh[k], v) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (t.has(k)) raw_store<TT, V>(dx + t.at(k), hv[k]);
    if (!y) continue;
    float s[2][TL::P];
#pragma unroll
    for (int q = 0; q < TL::P; ++q) s[0][q] = s[1][q] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!t.has(k)) continue;
      float w1[A], sg[A], gt[A], z1[A];
      t.param(j.w1, k, 1.f, w1);
      t.both(k, sg);
      if (TOK) {
        // scale and gate apart: dgate leaves here, the sums are weighted with the gate
        t.param(j.scale, k, 1.f, z1);
#pragma unroll
        for (int v = 0; v < A; ++v) gt[v] = j.gate ? __ldg(HND_G(j.gate + t.b * j.C + t.chan(k) + v)) : 1.f;
      }
      float b1[A];
      if (TOK) t.param(j.b1, k, 0.f, b1);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int q = TL::slot(v);
        // a dropped value reaches no sum, whatever it is: 0 times an infinity would
        const bool kept = keep[k] >> v & 1u;
        const float yh = kept ? (raw_at(ry[k], v) - mu1[q]) * rho1[q] : 0.f;
        const float md = kept ? hv[k][v] * j.factor : 0.f;
        if (TOK) {
          if (dgate) *HND_G(dgate + t.b * j.C + t.chan(k) + v) = z1[v] * md * (w1[v] * yh + b1[v]);
          acc[k][HND_PV(v)].x += gt[v] * md * yh;
          acc[k][HND_PV(v)].y += gt[v] * md;
        } else {
          acc[k][0].x += md * yh;
          acc[k][0].y += md;
        }
        hv[k][v] = md * sg[HND_PV(v)] * w1[HND_PV(v)];      // e from here on
        s[0][q] += hv[k][v];
        s[1][q] += hv[k][v] * yh;
      }
    }
    if (j.post) t.template sum<2>(s);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!t.has(k)) continue;
      if (j.post)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int q = TL::slot(v);
          const float yh = (raw_at(ry[k], v) - mu1[q]) * rho1[q];
          hv[k][v] = rho1[q] * (hv[k][v] - (j.post == 2 ? s[0][q] * inv : 0.f) - yh * (s[1][q] * inv));
        }
      raw_store<TT, V>(dy + t.at(k), hv[k]);
    }
  }
  if (!part) return;
  t.live = true;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int a = 0; a < A; ++a) {
      float4 s = acc[k][a];
      if (!TOK)
        for (int o = w / 2; o > 0; o >>= 1) {
          s.x += __shfl_xor_sync(0xFFFFFFFFu, s.x, o);
          s.y += __shfl_xor_sync(0xFFFFFFFFu, s.y, o);
          s.z += __shfl_xor_sync(0xFFFFFFFFu, s.z, o);
          s.w += __shfl_xor_sync(0xFFFFFFFFu, s.w, o);
        }
      if (t.has(k) && (TOK || t.lane == 0)) {
        const long long row = TOK ? blockIdx.x * static_cast<long long>(t.groups) + t.cg : blockIdx.x;
        *HND_G(part + row * j.C + t.chan(k) + a) = s;
      }
    }
}

}  // namespace hnd
