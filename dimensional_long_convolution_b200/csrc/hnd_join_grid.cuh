// hnd_join_grid.cuh -- the join on aligned grids: persistent blocks that bring
// the next tile while they work on this one.
//
// What hnd_join.cuh does in registers alone is held back by its loads: a block
// waits for its tile, works, stores, and the two blocks an SM has room for
// leave memory idle in between (2 x 128 x 256^2 bf16 forward: 87 us, a quarter
// of the bandwidth).  Here a thread copies its own vectors of the next tile
// into its own slots of shared memory (cp.async, 16 bytes each) as soon as
// this tile's are used up.  No other thread reads the slots, so no barrier
// guards them.  Arithmetic runs on pairs of positions (two fp32 operations an
// instruction), and the per-channel factors lie in shared memory for the whole
// run of the block.
//
// W neighbouring lanes hold 16 bytes of positions each, the rest of the 256
// threads the channels, K apiece.
#pragma once

#include "hnd_div.cuh"
#include "hnd_join.cuh"

namespace hnd {
namespace grid {

constexpr int kT = 256;
constexpr int kWarps = kT / 32;

// ------------------------------------------------------------- pairs of fp32
__device__ __forceinline__ uint64_t as64(float2 v) { return *reinterpret_cast<const uint64_t*>(&v); }
__device__ __forceinline__ float2 as2(uint64_t v) { return *reinterpret_cast<const float2*>(&v); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 add(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as64(a)), "l"(as64(b)));
  return as2(r);
}
__device__ __forceinline__ float2 mul(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as64(a)), "l"(as64(b)));
  return as2(r);
}
__device__ __forceinline__ float2 fma(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(as64(a)), "l"(as64(b)), "l"(as64(c)));
  return as2(r);
}

// 16 bytes as pairs: 4 of bf16, 2 of fp32.
template <class TT>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int Q = 4;
  static __device__ __forceinline__ float2 get(const uint4& u, int q) {
    const uint32_t w = q == 0 ? u.x : q == 1 ? u.y : q == 2 ? u.z : u.w;
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint4 put(const float2 (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[q].x, f[q].y);
      w[q] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<float> {
  static constexpr int Q = 2;
  static __device__ __forceinline__ float2 get(const uint4& u, int q) {
    return q == 0 ? make_float2(__uint_as_float(u.x), __uint_as_float(u.y))
                  : make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ uint4 put(const float2 (&f)[2]) {
    return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                      __float_as_uint(f[1].y));
  }
};

__device__ __forceinline__ void copy16(uint4* slot, const void* src) {
  if (HND_RANGE_OK(src, 16))
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(slot))),
                 "l"(src)
                 : "memory");
}
__device__ __forceinline__ void copies_done() {
  asm volatile("cp.async.commit_group;\n cp.async.wait_group 0;" ::: "memory");
}

// Shared memory: slots [tensor][K][kT] of 16 bytes, factors [C], sums.
inline size_t smem_bytes(int tensors, int K, long long C, int w, int V) {
  return static_cast<size_t>(tensors) * K * kT * 16 + static_cast<size_t>(C) * 16 + sizeof(float) * (kWarps + 1) * 2 * w * V;
}

// Where a thread's vectors of a tile lie: its first element, its sample, and a
// bit for each of its channels that is there.
struct Spot {
  long long at;
  int b;
  unsigned on;
};

template <class TT, int K>
struct Grid {
  static constexpr int Q = Vec<TT>::Q, V = 2 * Q;
  const JoinDev& j;
  const int w, lane, cg, rows, C;
  unsigned chans = 0;               // bit k: channel k of the thread exists
  long long own, step;              // of its first channel in a sample, and from one of its channels to the next
  uint4* slots;
  float4* coef;                     // of a channel: scale w1, scale b1, w2, b2
  float* part;                      // [kWarps][2 V w]
  float* total;                     // [2 V w]

  __device__ Grid(const JoinDev& jj, int lanes, int tensors, unsigned char* smem)
      : j(jj), w(lanes), lane(threadIdx.x % lanes), cg(threadIdx.x / lanes), rows(kT / lanes), C(static_cast<int>(jj.C)) {
#pragma unroll
    for (int k = 0; k < K; ++k) chans |= static_cast<unsigned>(chan(k) < C) << k;
    own = cg * j.L;
    step = rows * j.L;
    slots = reinterpret_cast<uint4*>(smem) + threadIdx.x;
    coef = reinterpret_cast<float4*>(reinterpret_cast<uint4*>(smem) + tensors * K * kT);
    part = reinterpret_cast<float*>(coef + C);
    total = part + kWarps * 2 * V * w;
    for (int c = threadIdx.x; c < C; c += kT) {
      const float sc = j.scale ? __ldg(HND_G(j.scale + c)) : 1.f;
      *HND_S(coef + c) = make_float4(sc * (j.w1 ? __ldg(HND_G(j.w1 + c)) : 1.f), sc * (j.b1 ? __ldg(HND_G(j.b1 + c)) : 0.f),
                                     j.w2 ? __ldg(HND_G(j.w2 + c)) : 1.f, j.b2 ? __ldg(HND_G(j.b2 + c)) : 0.f);
    }
    __syncthreads();
  }
  __device__ int chan(int k) const { return cg + k * rows; }
  __device__ uint4 raw(int tensor, int k) const { return *HND_S(slots + (tensor * K + k) * kT); }
  __device__ float gate(const Spot& s, int k) const {
    return j.gate ? __ldg(HND_G(j.gate + static_cast<long long>(s.b) * C + chan(k))) : 1.f;
  }
  // Vector u of sample b.
  __device__ Spot spot(int b, int u, bool live) const {
    return Spot{live ? b * j.C * j.L + static_cast<long long>(u) * V + own : 0, live ? b : 0, live ? chans : 0u};
  }
  __device__ void fetch(const Spot& s, int tensor, const TT* p) const {
    if (!p) return;
    const TT* from = p + s.at;
#pragma unroll
    for (int k = 0; k < K; ++k, from += step)
      if (s.on >> k & 1u) copy16(slots + (tensor * K + k) * kT, from);
  }
  __device__ void store(const Spot& s, TT* p, int k, const float2 (&f)[Q]) const {
    __stcs(HND_G(reinterpret_cast<uint4*>(p + (s.at + k * step))), Vec<TT>::put(f));
  }

  // Sums over the channels of N values at each of the thread's positions:
  // over the warp's channel rows by shuffles, over the warps by the first
  // W V N threads, each for one value.
  template <int N>
  __device__ void sum(float2 (&s)[N][Q]) const {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int q = 0; q < Q; ++q)
        for (int o = 16; o >= w; o >>= 1) {
          float2 t;
          t.x = __shfl_xor_sync(0xFFFFFFFFu, s[n][q].x, o);
          t.y = __shfl_xor_sync(0xFFFFFFFFu, s[n][q].y, o);
          s[n][q] = add(s[n][q], t);
        }
    constexpr int NV = N * V;
    const int warp = threadIdx.x / 32, values = w * NV;
    if ((threadIdx.x & 31) < w)
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int q = 0; q < Q; ++q)
          *HND_S(reinterpret_cast<float2*>(part + warp * 2 * V * w + lane * NV + n * V + 2 * q)) = s[n][q];
    __syncthreads();
    for (int v = threadIdx.x; v < values; v += kT) {
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) t += *HND_S(part + i * 2 * V * w + v);
      *HND_S(total + v) = t;
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int q = 0; q < Q; ++q) s[n][q] = *HND_S(reinterpret_cast<const float2*>(total + lane * NV + n * V + 2 * q));
  }
  // Mean (negative) and reciprocal deviation of f(k, q) at each position.
  template <class Fn>
  __device__ void stats(const Spot& at, int kind, float eps, float2 (&neg)[Q], float2 (&rho)[Q], Fn f) const {
#pragma unroll
    for (int q = 0; q < Q; ++q) neg[q] = both(0.f), rho[q] = both(1.f);
    if (!kind) return;
    const float inv = 1.f / static_cast<float>(j.C);
    float2 s[1][Q];
    if (kind == 2) {
#pragma unroll
      for (int q = 0; q < Q; ++q) s[0][q] = both(0.f);
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (at.on >> k & 1u) f(k, [&](int q, float2 v) { s[0][q] = add(s[0][q], v); });
      sum(s);
#pragma unroll
      for (int q = 0; q < Q; ++q) neg[q] = mul(s[0][q], both(-inv));
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) s[0][q] = both(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (at.on >> k & 1u)
        f(k, [&](int q, float2 v) {
          const float2 d = add(v, neg[q]);
          s[0][q] = fma(d, d, s[0][q]);
        });
    sum(s);
#pragma unroll
    for (int q = 0; q < Q; ++q)
      rho[q] = make_float2(rsqrtf(s[0][q].x * inv + eps), rsqrtf(s[0][q].y * inv + eps));
  }

  // y's statistics, the dropout bits and h.  Slots: 0 x, 1 y.
  __device__ void head(const Spot& at, bool has_y, unsigned (&keep)[K], float2 (&hv)[K][Q], float2 (&neg)[Q], float2 (&rho)[Q]) const {
    if (!has_y) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (at.on >> k & 1u) {
          const uint4 x = raw(0, k);
#pragma unroll
          for (int q = 0; q < Q; ++q) hv[k][q] = Vec<TT>::get(x, q);
        }
      return;
    }
    stats(at, j.post, j.eps1, neg, rho, [&](int k, auto use) {
      const uint4 y = raw(1, k);
#pragma unroll
      for (int q = 0; q < Q; ++q) use(q, Vec<TT>::get(y, q));
    });
    if (j.border) {
      const DropState ds = drop_state(j.rng);
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (at.on >> k & 1u) keep[k] = keep_bits<V>(ds, j.border, at.at + k * step);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!(at.on >> k & 1u)) continue;
      const uint4 x = raw(0, k), y = raw(1, k);
      const float4 cf = *HND_S(coef + chan(k));
      const float g = gate(at, k) * j.factor;
      const float2 al = both(cf.x * g), be = both(cf.y * g);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const float2 xv = Vec<TT>::get(x, q);
        float2 v = fma(mul(add(Vec<TT>::get(y, q), neg[q]), rho[q]), al, be);
        if (j.border) {
          v.x = (keep[k] >> (2 * q) & 1u) ? v.x : 0.f;
          v.y = (keep[k] >> (2 * q + 1) & 1u) ? v.y : 0.f;
        }
        hv[k][q] = add(xv, v);
      }
    }
  }
};

template <class TT, int K>
__global__ void __launch_bounds__(kT, 3) k_join_grid_fwd(const JoinDev j, int w, Div per, int units,
                                                         const TT* __restrict__ x, const TT* __restrict__ y,
                                                         TT* __restrict__ h, TT* __restrict__ n) {
  extern __shared__ __align__(16) unsigned char hnd_dyn_smem[];
  using G = Grid<TT, K>;
  constexpr int Q = G::Q;
  const G t(j, w, 2, hnd_dyn_smem);
  // vectors of positions are counted through the samples; `per` is those of one
  auto spot = [&](int u) {
    const int b = per.quot(u);
    return t.spot(b, u - b * static_cast<int>(per.d), u < units);
  };
  const int stride = gridDim.x * w;
  int u = blockIdx.x * w + t.lane;
  Spot at = spot(u);
  t.fetch(at, 0, x);
  t.fetch(at, 1, y);
  for (; u - t.lane < units; u += stride) {
    copies_done();
    unsigned keep[K];
    float2 hv[K][Q], neg[Q], rho[Q];
    t.head(at, y != nullptr, keep, hv, neg, rho);
    // the slots are used up: on to the next tile's copies
    const Spot next = spot(u + stride);
    t.fetch(next, 0, x);
    t.fetch(next, 1, y);
    if (h)
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (at.on >> k & 1u) t.store(at, h, k, hv[k]);
    if (n) {
      t.stats(at, j.pre, j.eps2, neg, rho, [&](int k, auto use) {
#pragma unroll
        for (int q = 0; q < Q; ++q) use(q, hv[k][q]);
      });
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!(at.on >> k & 1u)) continue;
        const float4 cf = *HND_S(t.coef + t.chan(k));
#pragma unroll
        for (int q = 0; q < Q; ++q) hv[k][q] = fma(mul(add(hv[k][q], neg[q]), rho[q]), both(cf.z), both(cf.w));
        t.store(at, n, k, hv[k]);
      }
    }
    at = next;
  }
}

// Gradients: a block goes through the tiles of its chunk of a sample and
// leaves each channel's sums of dht m yhat, dht m, dn hhat and dn in
// part[block][C].
template <class TT, int K>
__global__ void __launch_bounds__(kT, 2)
    k_join_grid_bwd(const JoinDev j, int w, int per, int chunks, const TT* __restrict__ x, const TT* __restrict__ y,
                    const TT* __restrict__ dh, const TT* __restrict__ dn, TT* __restrict__ dx, TT* __restrict__ dy,
                    float4* __restrict__ part) {
  extern __shared__ __align__(16) unsigned char hnd_dyn_smem[];
  using G = Grid<TT, K>;
  constexpr int Q = G::Q;
  const G t(j, w, 4, hnd_dyn_smem);
  const float2 inv = both(1.f / static_cast<float>(j.C));
  const int sample = blockIdx.x / chunks, stride = chunks * w;
  float4 acc[K];
#pragma unroll
  for (int k = 0; k < K; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto spot = [&](int u) { return t.spot(sample, u, u < per); };
  int u = (blockIdx.x - sample * chunks) * w + t.lane;
  Spot at = spot(u);
  t.fetch(at, 0, x);
  t.fetch(at, 1, y);
  t.fetch(at, 2, dn);
  t.fetch(at, 3, dh);
  for (; u - t.lane < per; u += stride) {
    copies_done();
    unsigned keep[K];
    float2 hv[K][Q], neg1[Q], rho1[Q], neg2[Q], rho2[Q];
    t.head(at, y != nullptr, keep, hv, neg1, rho1);
    const Spot next = spot(u + stride);      // used-up slots take the next tile
    t.fetch(next, 0, x);
    if (dn) {
      t.stats(at, j.pre, j.eps2, neg2, rho2, [&](int k, auto use) {
#pragma unroll
        for (int q = 0; q < Q; ++q) use(q, hv[k][q]);
      });
      float2 s[2][Q];
#pragma unroll
      for (int q = 0; q < Q; ++q) s[0][q] = s[1][q] = both(0.f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!(at.on >> k & 1u)) continue;
        const uint4 rn = t.raw(2, k);
        const float2 w2 = both((*HND_S(t.coef + t.chan(k))).z);
        float2 z = both(0.f), u = both(0.f);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const float2 d = Vec<TT>::get(rn, q), a = mul(d, w2);
          hv[k][q] = mul(add(hv[k][q], neg2[q]), rho2[q]);      // hhat from here on
          s[0][q] = add(s[0][q], a);
          s[1][q] = fma(a, hv[k][q], s[1][q]);
          z = fma(d, hv[k][q], z);
          u = add(u, d);
        }
        acc[k].z += z.x + z.y;
        acc[k].w += u.x + u.y;
      }
      t.template sum<2>(s);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        s[0][q] = j.pre == 2 ? mul(s[0][q], mul(inv, both(-1.f))) : both(0.f);
        s[1][q] = mul(s[1][q], mul(inv, both(-1.f)));
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!(at.on >> k & 1u)) continue;
        const uint4 rn = t.raw(2, k);
        uint4 rh = make_uint4(0, 0, 0, 0);
        if (dh) rh = t.raw(3, k);
        const float2 w2 = both((*HND_S(t.coef + t.chan(k))).z);
#pragma unroll
        for (int q = 0; q < Q; ++q)      // dht from here on
          hv[k][q] = fma(rho2[q], fma(hv[k][q], s[1][q], fma(Vec<TT>::get(rn, q), w2, s[0][q])), Vec<TT>::get(rh, q));
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        uint4 rh = make_uint4(0, 0, 0, 0);
        if (dh && (at.on >> k & 1u)) rh = t.raw(3, k);
#pragma unroll
        for (int q = 0; q < Q; ++q) hv[k][q] = Vec<TT>::get(rh, q);
      }
    }
    t.fetch(next, 2, dn);
    t.fetch(next, 3, dh);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (at.on >> k & 1u) t.store(at, dx, k, hv[k]);
    if (y) {
      float2 s[2][Q];
#pragma unroll
      for (int q = 0; q < Q; ++q) s[0][q] = s[1][q] = both(0.f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!(at.on >> k & 1u)) continue;
        const uint4 ry = t.raw(1, k);
        const float2 al = both((*HND_S(t.coef + t.chan(k))).x * t.gate(at, k));
        float2 a = both(0.f), r = both(0.f);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const float2 yh = mul(add(Vec<TT>::get(ry, q), neg1[q]), rho1[q]);
          float2 md = mul(hv[k][q], both(j.factor));
          if (j.border) {
            md.x = (keep[k] >> (2 * q) & 1u) ? md.x : 0.f;
            md.y = (keep[k] >> (2 * q + 1) & 1u) ? md.y : 0.f;
          }
          a = fma(md, yh, a);
          r = add(r, md);
          hv[k][q] = mul(md, al);      // e from here on
          s[0][q] = add(s[0][q], hv[k][q]);
          s[1][q] = fma(hv[k][q], yh, s[1][q]);
        }
        acc[k].x += a.x + a.y;
        acc[k].y += r.x + r.y;
      }
      if (j.post) {
        t.template sum<2>(s);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          s[0][q] = j.post == 2 ? mul(s[0][q], mul(inv, both(-1.f))) : both(0.f);
          s[1][q] = mul(s[1][q], mul(inv, both(-1.f)));
        }
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!(at.on >> k & 1u)) continue;
        if (j.post) {
          const uint4 ry = t.raw(1, k);
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            const float2 yh = mul(add(Vec<TT>::get(ry, q), neg1[q]), rho1[q]);
            hv[k][q] = mul(rho1[q], fma(yh, s[1][q], add(hv[k][q], s[0][q])));
          }
        }
        t.store(at, dy, k, hv[k]);
      }
      t.fetch(next, 1, y);
    }
    at = next;
  }
  if (!part) return;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float4 s = acc[k];
    for (int o = w / 2; o > 0; o >>= 1) {
      s.x += __shfl_xor_sync(0xFFFFFFFFu, s.x, o);
      s.y += __shfl_xor_sync(0xFFFFFFFFu, s.y, o);
      s.z += __shfl_xor_sync(0xFFFFFFFFu, s.z, o);
      s.w += __shfl_xor_sync(0xFFFFFFFFu, s.w, o);
    }
    if ((t.chans >> k & 1u) && t.lane == 0) *HND_G(part + blockIdx.x * j.C + t.chan(k)) = s;
  }
}

}  // namespace grid
}  // namespace hnd
