// hnd_join_grid.cuh -- the join on grids: persistent blocks that bring the next
// tile while they work on this one.
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
// threads the channels, K apiece.  The loops over a thread's channels have no
// branches, so that the K of them overlap: a channel that does not exist has
// zeros in its slots and factors, and counts for nothing in a variance.
//
// Rows that do not start on 16 bytes (RAG) come as the aligned vectors that
// cover them, one more than the lanes, and every thread shifts its positions
// out of its own and the next one's; on the way out it shifts them back with
// the lane before, so that all but a row's first and last vector leave whole.
// Eight elements then take two counters of the generator; the second is the
// next lane's first.  (One value a thread and load, as hnd_join.cuh does it for
// such rows, took 107 us for 13 x 204 x 777 bf16 forward and backward, this 90.)
//
// 2 x 128 x 256^2 bf16 forward: 31 us.  8 x 256 x 64^2 fp32: forward 32 us,
// backward 67, bound by latency (51 and 42% of the issue slots).
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
  using Bits = unsigned short;
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
  using Bits = unsigned;
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

// 16 bytes, or the first `bytes` of them and zeros.
__device__ __forceinline__ void copy16(uint4* slot, const void* src, int bytes = 16) {
  if (HND_RANGE_OK(src, bytes))
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(slot))),
                 "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copies_done() {
  asm volatile("cp.async.commit_group;\n cp.async.wait_group 0;" ::: "memory");
}

// Elements n .. n + V - 1 of a and b one after the other (0 <= n < V).
template <class TT>
__device__ __forceinline__ uint4 funnel(const uint4& a, const uint4& b, unsigned n) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  const unsigned words = sizeof(TT) == 2 ? n >> 1 : n;
  if (words & 2)
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  if (words & 1)
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  if constexpr (sizeof(TT) == 2)
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (n & 1) * 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The first n elements, and zeros.
template <class TT>
__device__ __forceinline__ uint4 first(const uint4& a, int n) {
  uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if constexpr (sizeof(TT) == 2)
      w[i] = 2 * i + 1 < n ? w[i] : 2 * i < n ? w[i] & 0xFFFFu : 0u;
    else
      w[i] = i < n ? w[i] : 0u;
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The elements whose bits are set, one by one.
template <class TT>
__device__ __forceinline__ void put_some(TT* p, const uint4& a, unsigned bits) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < static_cast<int>(16 / sizeof(TT)); ++i)
    if (bits >> i & 1u) {
      if constexpr (sizeof(TT) == 2)
        *HND_G(reinterpret_cast<unsigned short*>(p) + i) = static_cast<unsigned short>(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
      else
        *HND_G(reinterpret_cast<unsigned*>(p) + i) = w[i];
    }
}

// Shared memory: slots [tensor][K][rows][w, and one more if ragged] of 16
// bytes, factors [K][rows], sums; ragged: [2][rows][2] vectors of row ends.
inline size_t smem_bytes(int tensors, int K, int w, int V, bool ragged) {
  const size_t rows = kT / w, slots = static_cast<size_t>(tensors) * K * (kT + (ragged ? rows : 0));
  return 16 * (slots + K * rows + (ragged ? 4 * rows : 0)) + sizeof(float) * (kWarps + 1) * 2 * w * V;
}

// Where a thread's vectors of a tile lie: its first element, its sample, a bit
// for each of its channels that is there, and how many of its positions are
// (ragged: whether the next lane has some, and whether all of the tile's are
// there).
struct Spot {
  long long at;
  int b;
  unsigned on;
  int n;
  bool next, inner;
};

// FIX: the block keeps to one sample, whose gate goes into the factors.
template <class TT, int K, bool RAG, bool FIX>
struct Grid {
  static constexpr int Q = Vec<TT>::Q, V = 2 * Q;
  const JoinDev& j;
  const int w, lane, cg, rows, C;
  unsigned chans = 0;               // bit k: channel k of the thread exists
  long long own, step;              // of its first channel in a sample, and from one of its channels to the next
  uint4* slots;                     // its own
  int pitch;                        // slots from one k to the next
  float4* coef;                     // of a channel: scale w1, scale b1 (times the gate, FIX), w2, b2
  DropState ds{};
  float* part;                      // [kWarps][2 V w]
  float* total;                     // [2 V w]
  uint4* ends;                      // ragged: of the thread's row, its first and last lane's vector, in turns
  mutable int turn = 0;

  __device__ Grid(const JoinDev& jj, int lanes, int tensors, unsigned char* smem, long long sample)
      : j(jj), w(lanes), lane(threadIdx.x % lanes), cg(threadIdx.x / lanes), rows(kT / lanes), C(static_cast<int>(jj.C)) {
#pragma unroll
    for (int k = 0; k < K; ++k) chans |= static_cast<unsigned>(chan(k) < C) << k;
    own = cg * j.L;
    step = rows * j.L;
    pitch = kT + (RAG ? rows : 0);
    slots = reinterpret_cast<uint4*>(smem) + cg * (w + RAG) + lane;
    coef = reinterpret_cast<float4*>(reinterpret_cast<uint4*>(smem) + tensors * K * pitch);
    part = reinterpret_cast<float*>(coef + K * rows);
    total = part + kWarps * 2 * V * w;
    ends = reinterpret_cast<uint4*>(total + 2 * V * w) + 2 * cg;
    for (int c = threadIdx.x; c < K * rows; c += kT) {
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < C) {
        float sc = j.scale ? __ldg(HND_G(j.scale + c)) : 1.f;
        if (FIX && j.gate) sc *= __ldg(HND_G(j.gate + sample * C + c));
        f.x = sc * (j.w1 ? __ldg(HND_G(j.w1 + c)) : 1.f);
        f.y = sc * (j.b1 ? __ldg(HND_G(j.b1 + c)) : 0.f);
        f.z = j.w2 ? __ldg(HND_G(j.w2 + c)) : 1.f;
        f.w = j.b2 ? __ldg(HND_G(j.b2 + c)) : 0.f;
      }
      *HND_S(coef + c) = f;
    }
    if (j.border) ds = drop_state(j.rng);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (!there(k))
        for (int i = 0; i < tensors; ++i)
          for (int e = 0; e < (RAG && lane == w - 1 ? 2 : 1); ++e)      // the row's extra slot too
            *HND_S(slots + (i * K + k) * pitch + e) = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
  __device__ int chan(int k) const { return cg + k * rows; }
  __device__ bool there(int k) const { return chans >> k & 1u; }
  __device__ uint4 raw(int tensor, int k) const { return *HND_S(slots + (tensor * K + k) * pitch); }
  __device__ float gate(const Spot& s, int k) const {
    return !FIX && j.gate && there(k) ? __ldg(HND_G(j.gate + static_cast<long long>(s.b) * C + chan(k))) : 1.f;
  }
  // Ragged: how far into its aligned vector the lane's first position lies.
  __device__ int shift(const Spot& s, int k) const {
    return static_cast<int>((static_cast<unsigned>(s.at) + k * static_cast<unsigned>(step)) & (V - 1));
  }
  // Vector u of sample b, `left` positions of the sample from there on.
  __device__ Spot spot(int b, int u, int left) const {
    const bool live = left > 0;
    return Spot{b * j.C * j.L + static_cast<long long>(u) * V + own, live ? b : 0, live ? chans : 0u,
                live ? min(left, V) : 0, RAG && lane + 1 < w && left > V, RAG && left >= (w - lane) * V};
  }
  __device__ void fetch(const Spot& s, int tensor, const TT* p) const {
    if (!p) return;
    if constexpr (RAG) {
      __syncwarp();      // the slot after the lane's own is another lane's
      const long long all = j.T * j.C;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!(s.on >> k & 1u)) continue;
        const int in = shift(s, k);
        const long long from = s.at + k * step - in, rest = (all - from) * static_cast<int>(sizeof(TT));
        uint4* slot = slots + (tensor * K + k) * pitch;
        copy16(slot, p + from, rest < 16 ? static_cast<int>(rest) : 16);
        if (!s.next && in + s.n > V)
          copy16(slot + 1, p + from + V, rest < 32 ? static_cast<int>(rest) - 16 : 16);
      }
    } else {
      const TT* from = p + s.at;
#pragma unroll
      for (int k = 0; k < K; ++k, from += step)
        if (s.on >> k & 1u) copy16(slots + (tensor * K + k) * pitch, from);
    }
  }
  // Ragged: the lane's own positions out of the aligned vectors, zeros behind
  // the row's end, back into its slots.
  __device__ void align(const Spot& s, int tensor) const {
    if constexpr (RAG) {
      uint4 v[K];
      __syncwarp();
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const uint4* slot = slots + (tensor * K + k) * pitch;
        v[k] = funnel<TT>(*HND_S(slot), *HND_S(slot + 1), shift(s, k));
        if (s.n < V) v[k] = first<TT>(v[k], s.n);
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < K; ++k) *HND_S(slots + (tensor * K + k) * pitch) = v[k];
    }
  }
  // All lanes of a warp take part, for each k.
  __device__ void store(const Spot& s, TT* p, int k, const float2 (&f)[Q]) const {
    const bool on = s.on >> k & 1u;
    const long long e = s.at + k * step;
    const uint4 mine = Vec<TT>::put(f);
    if constexpr (RAG) {
      const int at = shift(s, k);
      uint4 before;
      before.x = __shfl_up_sync(0xFFFFFFFFu, mine.x, 1, w);
      before.y = __shfl_up_sync(0xFFFFFFFFu, mine.y, 1, w);
      before.z = __shfl_up_sync(0xFFFFFFFFu, mine.z, 1, w);
      before.w = __shfl_up_sync(0xFFFFFFFFu, mine.w, 1, w);
      // the vector that the lane's first position lies in, and what spills into the one after it
      const uint4 head = at ? funnel<TT>(before, mine, V - at) : mine;
      TT* to = p + (e - at);
      if (s.inner) {
        // Whole vectors, but for a row's first and last, which lie in V elements of its first and last lane: element
        // i of the one or the other, by lane i.
        uint4* pair = ends + turn * 2 * rows;      // two turns: the one before last has been read
        turn ^= 1;
        if (lane == 0) *HND_S(pair) = mine;
        if (lane == w - 1) *HND_S(pair + 1) = mine;
        __syncwarp();
        if (on && (lane || !at)) __stcs(HND_G(reinterpret_cast<uint4*>(to)), head);
        using Bits = typename Vec<TT>::Bits;
        for (int i = lane; i < V; i += w) {
          const int last = i >= V - at;
          const Bits v = *HND_S(reinterpret_cast<const Bits*>(pair + last) + i);
          if (on && at) *HND_G(reinterpret_cast<Bits*>(p + (e - lane * V + last * (w - 1) * V + i))) = v;
        }
        return;
      }
      unsigned some = on ? (2u << min(V, at + s.n) - 1) - (lane ? 1u : 1u << at) : 0u;
      if (some == (1u << V) - 1) {
        __stcs(HND_G(reinterpret_cast<uint4*>(to)), head);
        some = 0;
      }
      // a row's first vector by one lane and its spill by another, in one go
      const unsigned over = on && !s.next && at + s.n > V ? (1u << (at + s.n - V)) - 1 : 0u;
      const uint4 tail = funnel<TT>(mine, mine, (V - at) & (V - 1));
      const bool spills = over && !some;
      put_some(spills ? to + V : to, spills ? tail : head, spills ? over : some);
      if (__any_sync(0xFFFFFFFFu, over && some)) put_some(to + V, tail, over && some ? over : 0u);
    } else {
      if (on) __stcs(HND_G(reinterpret_cast<uint4*>(p + e)), mine);
    }
  }

  // The eight mask bits of a group.
  __device__ unsigned group_bits(long long group) const {
    const uint4 v = drop_lots(ds, static_cast<uint64_t>(group));
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    unsigned bits = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      bits |= static_cast<unsigned>((u[i] & 0xFFFFu) >= j.border) << (2 * i) |
              static_cast<unsigned>((u[i] >> 16) >= j.border) << (2 * i + 1);
    return bits;
  }
  // keep[k]: a bit for each of the lane's positions.  All lanes take part.
  __device__ void mask(const Spot& s, unsigned (&keep)[K]) const {
    if constexpr (V == 8 && !RAG) {
#pragma unroll
      for (int k = 0; k < K; ++k) keep[k] = group_bits((s.at + k * step) >> 3);
    } else if constexpr (V == 8) {
      // lane i has group i of the row's tile; of the group behind the last lane's, lane q takes channel q / rows of a
      // warp in row q % rows
      const int rw = 32 / w, q = threadIdx.x & 31, row = q / w;
#pragma unroll
      for (int k = 0; k < K; ++k) keep[k] = group_bits((s.at + k * step) >> 3);
      unsigned behind[K];
      for (int done = 0; done < K * rw; done += 32) {
        const int k = (done + q) / rw, r = (done + q) % rw;
        const long long at0 = __shfl_sync(0xFFFFFFFFu, s.at, r * w + w - 1);      // of that row's last lane
        const unsigned got = k < K ? group_bits(((at0 + k * step) >> 3) + 1) : 0u;
#pragma unroll
        for (int i = 0; i < K; ++i) {
          const int from = i * rw + row - done;
          const unsigned v = __shfl_sync(0xFFFFFFFFu, got, from & 31);
          if (from >= 0 && from < 32) behind[i] = v;
        }
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        unsigned after = __shfl_down_sync(0xFFFFFFFFu, keep[k], 1, w);
        if (lane == w - 1) after = behind[k];
        keep[k] = (keep[k] | after << 8) >> shift(s, k);
      }
    } else if (!RAG && K % 2 == 0 && w > 1 && j.L % 8 == 0) {
      // two lanes lie in one group: each takes one channel of two
      const int odd = lane & 1;
#pragma unroll
      for (int k = 0; k + 1 < K; k += 2) {
        const unsigned mine = group_bits((s.at + (k + odd) * step) >> 3);
        const unsigned other = __shfl_xor_sync(0xFFFFFFFFu, mine, 1);
        keep[k] = (odd ? other : mine) >> (4 * odd);
        keep[k + 1] = (odd ? mine : other) >> (4 * odd);
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const long long e = s.at + k * step;
        unsigned bits = group_bits(e >> 3);
        if (RAG && (e & 7) > 4) bits |= group_bits((e >> 3) + 1) << 8;
        keep[k] = bits >> (e & 7);
      }
    }
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
  __device__ void stats(int kind, float eps, float2 (&neg)[Q], float2 (&rho)[Q], Fn f) const {
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
        f(k, [&](int q, float2 v) { s[0][q] = add(s[0][q], v); });
      sum(s);
#pragma unroll
      for (int q = 0; q < Q; ++q) neg[q] = mul(s[0][q], both(-inv));
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) s[0][q] = both(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const float2 counts = both(there(k) ? 1.f : 0.f);
      f(k, [&](int q, float2 v) {
        float2 d = v;
        if (kind == 2) d = mul(add(v, neg[q]), counts);
        s[0][q] = fma(d, d, s[0][q]);
      });
    }
    sum(s);
#pragma unroll
    for (int q = 0; q < Q; ++q)
      rho[q] = make_float2(rsqrtf(s[0][q].x * inv + eps), rsqrtf(s[0][q].y * inv + eps));
  }

  // y's statistics, the dropout bits and h.  Slots: 0 x, 1 y.
  __device__ void head(const Spot& at, bool has_y, unsigned (&keep)[K], float2 (&hv)[K][Q], float2 (&neg)[Q],
                       float2 (&rho)[Q]) const {
    if (!has_y) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const uint4 x = raw(0, k);
#pragma unroll
        for (int q = 0; q < Q; ++q) hv[k][q] = Vec<TT>::get(x, q);
      }
      return;
    }
    stats(j.post, j.eps1, neg, rho, [&](int k, auto use) {
      const uint4 y = raw(1, k);
#pragma unroll
      for (int q = 0; q < Q; ++q) use(q, Vec<TT>::get(y, q));
    });
    if (j.border) {
      mask(at, keep);
      joined<true>(at, keep, hv, neg, rho);
    } else {
      joined<false>(at, keep, hv, neg, rho);
    }
  }
  template <bool DROP>
  __device__ void joined(const Spot& at, const unsigned (&keep)[K], float2 (&hv)[K][Q], const float2 (&neg)[Q],
                         const float2 (&rho)[Q]) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const uint4 x = raw(0, k), y = raw(1, k);
      const float4 cf = *HND_S(coef + chan(k));
      const float g = gate(at, k) * j.factor;
      const float2 al = both(cf.x * g), be = both(cf.y * g);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        float2 v = fma(mul(add(Vec<TT>::get(y, q), neg[q]), rho[q]), al, be);
        if (DROP) v = kept(keep[k], q, v);
        hv[k][q] = add(Vec<TT>::get(x, q), v);
      }
    }
  }
  static __device__ float2 kept(unsigned bits, int q, float2 v) {
    return make_float2((bits >> (2 * q) & 1u) ? v.x : 0.f, (bits >> (2 * q + 1) & 1u) ? v.y : 0.f);
  }
};

template <class TT, int K, bool RAG>
__global__ void __launch_bounds__(kT, RAG ? 2 : 3) k_join_grid_fwd(const JoinDev j, int w, Div per, int units,
                                                         const TT* __restrict__ x, const TT* __restrict__ y,
                                                         TT* __restrict__ h, TT* __restrict__ n) {
  extern __shared__ __align__(16) unsigned char hnd_dyn_smem[];
  using G = Grid<TT, K, RAG, false>;
  constexpr int Q = G::Q;
  const G t(j, w, 2, hnd_dyn_smem, 0);
  // Vectors of positions are counted through the samples, `per` to each, and a
  // tile takes w of them; ragged, a tile keeps to one sample and `per` counts
  // its tiles.
  auto spot = [&](int i) {
    const int u = RAG ? i : i * w + t.lane, b = per.quot(min(u, units - 1)), v = u - b * static_cast<int>(per.d);
    const int from = RAG ? v * w + t.lane : v;
    return t.spot(b, from, u < units ? static_cast<int>(min(j.L - static_cast<long long>(from) * G::V, 1LL << 30)) : 0);
  };
  const int tiles = RAG ? units : (units + w - 1) / w;
  Spot at = spot(blockIdx.x);
  t.fetch(at, 0, x);
  t.fetch(at, 1, y);
  for (int i = blockIdx.x; i < tiles; i += gridDim.x) {
    copies_done();
    t.align(at, 0);
    if (y) t.align(at, 1);
    unsigned keep[K];
    float2 hv[K][Q], neg[Q], rho[Q];
    t.head(at, y != nullptr, keep, hv, neg, rho);
    // the slots are used up: on to the next tile's copies
    const Spot next = spot(min(i + static_cast<int>(gridDim.x), tiles));
    t.fetch(next, 0, x);
    t.fetch(next, 1, y);
    if (h)
#pragma unroll
      for (int k = 0; k < K; ++k)
        t.store(at, h, k, hv[k]);
    if (n) {
      t.stats(j.pre, j.eps2, neg, rho, [&](int k, auto use) {
#pragma unroll
        for (int q = 0; q < Q; ++q) use(q, hv[k][q]);
      });
#pragma unroll
      for (int k = 0; k < K; ++k) {
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
template <class TT, int K, bool RAG>
__global__ void __launch_bounds__(kT, 2)
    k_join_grid_bwd(const JoinDev j, int w, int per, int chunks, const TT* __restrict__ x, const TT* __restrict__ y,
                    const TT* __restrict__ dh, const TT* __restrict__ dn, TT* __restrict__ dx, TT* __restrict__ dy,
                    float4* __restrict__ part) {
  extern __shared__ __align__(16) unsigned char hnd_dyn_smem[];
  using G = Grid<TT, K, RAG, true>;
  constexpr int Q = G::Q;
  const int sample = blockIdx.x / chunks, stride = chunks * w;
  const G t(j, w, 4, hnd_dyn_smem, sample);
  const float2 inv = both(1.f / static_cast<float>(j.C));
  float4 acc[K];
#pragma unroll
  for (int k = 0; k < K; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto spot = [&](int u) {
    return t.spot(sample, min(u, per), static_cast<int>(min(j.L - static_cast<long long>(min(u, per)) * G::V, 1LL << 30)));
  };
  int u = (blockIdx.x - sample * chunks) * w + t.lane;
  Spot at = spot(u);
  t.fetch(at, 0, x);
  t.fetch(at, 1, y);
  t.fetch(at, 2, dn);
  t.fetch(at, 3, dh);
  for (; u - t.lane < per; u += stride) {
    copies_done();
    t.align(at, 0);
    if (y) t.align(at, 1);
    if (dn) t.align(at, 2);
    if (dh) t.align(at, 3);
    unsigned keep[K];
    float2 hv[K][Q], neg1[Q], rho1[Q], neg2[Q], rho2[Q];
    t.head(at, y != nullptr, keep, hv, neg1, rho1);
    const bool live = at.n > 0;
    const Spot next = spot(u + stride);      // used-up slots take the next tile
    t.fetch(next, 0, x);
    if (dn) {
      t.stats(j.pre, j.eps2, neg2, rho2, [&](int k, auto use) {
#pragma unroll
        for (int q = 0; q < Q; ++q) use(q, hv[k][q]);
      });
      float2 s[2][Q];
#pragma unroll
      for (int q = 0; q < Q; ++q) s[0][q] = s[1][q] = both(0.f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
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
        acc[k].z += live ? z.x + z.y : 0.f;
        acc[k].w += live ? u.x + u.y : 0.f;
      }
      t.template sum<2>(s);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        s[0][q] = j.pre == 2 ? mul(s[0][q], mul(inv, both(-1.f))) : both(0.f);
        s[1][q] = mul(s[1][q], mul(inv, both(-1.f)));
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
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
        if (dh) rh = t.raw(3, k);
#pragma unroll
        for (int q = 0; q < Q; ++q) hv[k][q] = Vec<TT>::get(rh, q);
      }
    }
    t.fetch(next, 2, dn);
    t.fetch(next, 3, dh);
#pragma unroll
    for (int k = 0; k < K; ++k)
      t.store(at, dx, k, hv[k]);
    if (y) {
      float2 s[2][Q];
#pragma unroll
      for (int q = 0; q < Q; ++q) s[0][q] = s[1][q] = both(0.f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const uint4 ry = t.raw(1, k);
        const float2 al = both((*HND_S(t.coef + t.chan(k))).x * t.gate(at, k));
        const unsigned bits = j.border ? keep[k] : ~0u;
        float2 a = both(0.f), r = both(0.f);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          // a dropped value reaches no sum, whatever it is: 0 times an infinity would
          const float2 yh = G::kept(bits, q, mul(add(Vec<TT>::get(ry, q), neg1[q]), rho1[q]));
          const float2 md = G::kept(bits, q, mul(hv[k][q], both(j.factor)));
          a = fma(md, yh, a);
          r = add(r, md);
          hv[k][q] = mul(md, al);      // e from here on
          s[0][q] = add(s[0][q], hv[k][q]);
          s[1][q] = fma(hv[k][q], yh, s[1][q]);
        }
        acc[k].x += live ? a.x + a.y : 0.f;
        acc[k].y += live ? r.x + r.y : 0.f;
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
    if (t.there(k) && t.lane == 0) *HND_G(part + blockIdx.x * j.C + t.chan(k)) = s;
  }
}

}  // namespace grid
}  // namespace hnd
