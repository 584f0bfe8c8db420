// hnd_ffn_gemm.cuh -- the matrix products of the gated feed-forward block on
// the fifth-generation tensor cores, with the block's activation in their
// epilogues.
//
// Every product is D(m, n) = sum_k A(m, k) B(k, n); m lies in the lanes of
// tensor memory and n in its columns.  Operands keep the layout they have in
// memory: a tile whose m (or n) axis is the contiguous one is staged
// "MN-major", otherwise "K-major"; both in 128-byte swizzled shared memory,
// brought by TMA, whose out-of-range zeros cover every ragged edge.  Where m
// is the contiguous axis of D (positions of [B, C, L] outputs, channels of a
// weight gradient) a warp's stores of one n are adjacent; the hidden
// activations, which only these products read, lie the other way, [position]
// [channel], so that a thread has neighbouring channels to pack and store.
//
// A pair of CTAs computes a 256 x 256 tile (cta_group::2): each holds 128 rows
// of A, half of B's columns and 128 accumulator lanes.  One warp issues TMA,
// one (of the leading CTA) the MMAs, eight (sixteen for the bf16 hidden
// gradients) read the accumulators back.  Accumulators are fp32 in tensor
// memory, two of 256 columns, so that the epilogue of a tile runs under the
// products of the next.  A stage of four MMAs took 537 cycles with 160 and 96
// columns, about what 256 need, so every product has 256 where it can: G and U of 128 hidden channels side by side,
// and where the epilogue needs dH too, dH of 256 hidden channels in one half of
// tensor memory while their G and U pass through the other in two turns.
// (Tiles of 80 channels, 80 + 80 + 96 columns in each of two accumulators,
// overlap the epilogue: 75 us at C 256, F 1024 and 32768 positions, as here,
// but 506 against 440 us at C 2048, F 5632 and 8192.)  The hidden product at
// the first size takes 32 us, the second 19, the gradient dx 36, the weight
// gradients 52; the hidden product at the second 237 us, 1.6 PFLOP/s.
//
// Hidden activations are rounded to bf16 once, as the second product's
// operand: its tensor-core type, and half the bytes.  It makes the result's
// relative error 2.3e-3 where one rounding alone gives 1.7e-3.
//
// fp32 operands come as three bf16 planes (high, middle, low: 24 bits) and
// every K loop runs over the six plane products that reach 2^-24, the small
// ones first.  The tensor core truncates where it adds to an accumulator, a
// loss that grows with the number of additions (measured: 1.0e-6 of the
// result at depth 528, 1.4e-6 further on), so a loop is cut into pieces of
// 256 whose sums the epilogue adds up to the nearest: in the other half of
// tensor memory, or for the three hidden gradients in registers.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <type_traits>

#include "hnd_bounds.cuh"
#include "hnd_div.cuh"

namespace hnd {
namespace ffn {

constexpr int kBK = 64;                // depth of a stage
constexpr int kHalf = 128 * kBK * 2;   // bytes of A (and of B) per CTA and stage
constexpr int kStage = 2 * kHalf;

// One stretch of a K loop.
struct Seg {
  int a, b0, b1;             // tensor maps; b1 is the second CTA's B
  int a_mn, b_mn;            // 1: the tile's m (n) axis is contiguous in memory
  int a_batched, b_batched;  // the map's third coordinate follows the batch
  int ncols;                 // columns over the pair, at most 256
  int nstep, noff, nbase;    // n from tile to tile, to the second CTA's part, and of the tile's first
  int acc;                   // first accumulator column
  int clear;                 // starts this accumulator
};

enum OutKind {
  kOutTma = 0,      // bf16 by TMA
  kOutBf16 = 1,     // bf16, a lane's elements one by one
  kOutF32 = 2,      // the same in fp32
  kOutTok = 3       // token-major: a lane's columns are adjacent
};

// One product: tiles [batches][mt][nt][splits].
struct Job {
  int seg0, nseg;
  int batches, mt, nt, splits;
  int kbatches, kblocks;     // the K loop: batches (of weight gradients), stages of each
  int kper;                  // stages of a split
  // tiles of a split, tiles of eight m tiles, mt: with plain divisions the
  // issuing warps took longer to find a short tile than its products do
  Div per, group8, mdiv;
  long long M, N;            // extents of D
  int cols;                  // columns of a tile of kEpiOut: 256, 128 or 64
  int kind, map;             // how D leaves, and the map of kOutTma
  void* ptr;                 // D otherwise: element (m, n) of split s and batch b at
  long long bs, rs;          //   (s batches + b) bs + n rs + m, or with group > 0 at
  long long group, gs;       //   (m / group) gs + n rs + m % group; kOutTok: m rs + n
};

constexpr int kMaxMaps = 10, kMaxSegs = 3, kMaxJobs = 3;

struct Params {
  CUtensorMap map[kMaxMaps];
  Seg seg[kMaxSegs];
  Job job[kMaxJobs];
  int tiles;
  int a_plane, b_plane;      // third-coordinate distance of the planes
  int act;
  int piece;                 // fp32: stages of each segment that the tensor core adds up
  // the hidden tensors [plane][batch][position][channel]
  __nv_bfloat16* hid[3];
  long long hid_plane, hid_rs;
  int hmap[3];               // bf16: their maps
  int* status;
};

enum Epi { kEpiOut = 0, kEpiHidden = 1, kEpiGrad = 2 };

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ uint32_t s32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of the same shared location in the pair's leading CTA.
__device__ __forceinline__ uint32_t in_leader(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
// One lane of a converged warp.
__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Waits for a phase; after two seconds records a timeout and gives up.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, int* status) {
  if (bar_try(bar, parity)) return true;
  const uint64_t t0 = now_ns();
  for (;;) {
    for (int i = 0; i < 32; ++i)
      if (bar_try(bar, parity)) return true;
    if (now_ns() - t0 > 2000000000ull) break;
  }
  if (status) atomicCAS(status, 0, 6 /* HYENA_ND_ERR_DEVICE_TIMEOUT */);
  return false;
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Arrives at a barrier of the pair's other CTA.  Only tensor-memory reads come
// before it, which tcgen05.wait and fence order; release at cluster scope
// would wait for this thread's stores to memory too (2000 cycles a tile).
__device__ __forceinline__ void bar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map), "r"(src),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
// Arrives on the barrier at this offset in both CTAs once the MMAs so far are done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t (&r)[N], uint32_t addr);
template <>
__device__ __forceinline__ void tmem_load<32>(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, "
      "%24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
template <>
__device__ __forceinline__ void tmem_load<16>(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, "
      "%25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool named_all(int id, int threads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n barrier.cta.red.and.pred q, %1, %2, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(v ? 1u : 0u)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Shared-memory operand descriptor, 128-byte swizzle.  K-major: rows of 64 k,
// eight rows 1024 bytes apart.  MN-major: rows of 64 m (n), one row a k; eight
// rows 1024 bytes apart (stride offset), the next 64 m 8192 bytes on (leading
// offset).
__device__ __forceinline__ uint64_t operand(uint32_t addr, int mn) {
  const uint64_t lead = mn ? 8192 >> 4 : 1, stride = 1024 >> 4;
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | lead << 16 | stride << 32 | 1ull << 46 | 2ull << 61;
}
// bf16 x bf16 -> fp32, 256 x ncols over the pair.
__device__ __forceinline__ uint32_t instruction(int a_mn, int b_mn, int ncols) {
  return 1u << 4 | 1u << 7 | 1u << 10 | static_cast<uint32_t>(a_mn) << 15 | static_cast<uint32_t>(b_mn) << 16 |
         static_cast<uint32_t>(ncols >> 3) << 17 | static_cast<uint32_t>(256 >> 4) << 24;
}

// --------------------------------------------------------------- activation
constexpr float kInvSqrt2Pi = 0.39894228040143268f, kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float recip_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair64(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float (&o)[2]) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o[0]), "=f"(o[1]) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// 1 / (1 + exp(-g)) of two gates, from w = exp(-|g|) <= 1: 1 / (1 + w) above
// zero and w / (1 + w) below, which keeps its relative accuracy down to the
// smallest normal number (g s u may be large all the same) and is 0 beyond.
// bf16: one reciprocal of the product of the denominators, 4 at most, serves
// both, since the special-function unit (two exponentials and two reciprocals
// for a pair otherwise) is what the epilogue waits for.  A NaN comes back as
// 1/2, so that the other gate keeps its value, and is one again in the product
// with g.
template <bool F32>
__device__ __forceinline__ void sigmoid2(const float (&g)[2], float (&s)[2]) {
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float w = expf(-fabsf(g[i])), r = recip_fast(1.f + w);     // off by one unit in the last place at most
      s[i] = g[i] < 0.f ? w * r : r;
    }
  } else {
    float x[2], w[2];
    unpair(mul2(pair64(g[0], g[1]), pair64(-kLog2e, -kLog2e)), x);
#pragma unroll
    for (int i = 0; i < 2; ++i) w[i] = exp2_fast(fminf(-fabsf(x[i]), 0.f));
    const float d0 = 1.f + w[0], d1 = 1.f + w[1], r = recip_fast(d0 * d1), t[2] = {r * d1, r * d0};
#pragma unroll
    for (int i = 0; i < 2; ++i) s[i] = g[i] < 0.f ? w[i] * t[i] : t[i];
  }
}

// The normal distribution function Phi of two gates and e = exp(-g^2/2), which
// the slope needs too.  Below zero Phi keeps its relative accuracy (1/2 +
// erf/2 loses all of it from -5 on, and g Phi(g) u may be large all the same):
// Phi(-z) = e M(z), where M falls slowly from 1/2 like 1 / (z sqrt(2 pi)), and
// M = t P(t) in t = 1 / (1 + 0.35 z), P fitted over 0 <= z <= 16 for the least
// greatest relative error (a linear program on M = erfcx(z / sqrt 2) / 2):
// 3.2e-8 at degree 8.  bf16 takes it too, since the slope crosses zero at
// -0.75 and would keep an absolute error there (degree 4 has 7.2e-5).  Beyond
// 16, e is 0 in fp32, so that z may be cut at 64, which keeps z^2 and the
// product of both denominators finite; one reciprocal serves both gates.  A
// NaN comes back as 1 and is one again in the product with g.
template <bool F32>
__device__ __forceinline__ void normal2(const float (&g)[2], float (&cdf)[2], float (&e)[2]) {
  constexpr float a = 0.35f;
  constexpr float c[9] = {0.139621243f, 0.139864534f,  0.11981415f, 0.105579965f,  -0.0232757367f,
                          0.159409821f, -0.255916387f, 0.14406772f, -0.0291653275f};
  float z[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    z[i] = fminf(fabsf(g[i]), 64.f);
    if constexpr (F32) {      // exp of the whole square: its rounding counts z^2 / 2 times
      const float zz = z[i] * z[i], x = expf(-0.5f * zz);
      e[i] = fmaf(x, -0.5f * fmaf(z[i], z[i], -zz), x);
    } else {
      e[i] = exp2_fast(-0.5f * kLog2e * z[i] * z[i]);
    }
  }
  const float d0 = fmaf(a, z[0], 1.f), d1 = fmaf(a, z[1], 1.f), r = recip_fast(d0 * d1);
  const float t[2] = {r * d1, r * d0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float q = c[8];
#pragma unroll
    for (int k = 7; k >= 0; --k) q = fmaf(q, t[i], c[k]);
    q *= t[i] * e[i];
    cdf[i] = g[i] < 0.f ? q : 1.f - q;
  }
}

// act(g) u of two hidden channels.
template <bool F32, int ACT>
__device__ __forceinline__ void hidden2(const float (&g)[2], const float (&u)[2], float (&h)[2]) {
  float s[2];
  if constexpr (ACT == 0) {
    sigmoid2<F32>(g, s);
  } else {
    float e[2];
    normal2<F32>(g, s, e);
  }
  unpair(mul2(mul2(pair64(g[0], g[1]), pair64(s[0], s[1])), pair64(u[0], u[1])), h);
}

// H, dG and dU of two hidden channels.
template <bool F32, int ACT>
__device__ __forceinline__ void hidden_grads2(const float (&g)[2], const float (&u)[2], const float (&d)[2],
                                              float (&h)[2], float (&dg)[2], float (&du)[2]) {
  float s[2], e[2];
  if constexpr (ACT == 0)
    sigmoid2<F32>(g, s);
  else
    normal2<F32>(g, s, e);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float a = g[i] * s[i], da = ACT ? fmaf(g[i] * kInvSqrt2Pi, e[i], s[i]) : fmaf(a, 1.f - s[i], s[i]);
    h[i] = a * u[i];
    dg[i] = d[i] * u[i] * da;
    du[i] = d[i] * a;
  }
}

// The bf16 planes of an fp32 value.  Values beyond bf16's largest keep a
// finite high plane.
__device__ __forceinline__ void split3(float v, __nv_bfloat16& hi, __nv_bfloat16& mid, __nv_bfloat16& lo) {
  hi = __float2bfloat16_rn(v);
  if (fabsf(__bfloat162float(hi)) > 3.4e38f && fabsf(v) <= 3.4028235e38f) hi = __float2bfloat16_rz(v);
  const float r = v - __bfloat162float(hi);
  mid = __float2bfloat16_rn(r);
  lo = __float2bfloat16_rn(r - __bfloat162float(mid));
}

// Two values' planes, packed plane by plane.
__device__ __forceinline__ void split3x2(float a, float b, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  __nv_bfloat162 h[3];
  split3(a, h[0].x, h[1].x, h[2].x);
  split3(b, h[0].y, h[1].y, h[2].y);
  hi = *reinterpret_cast<const uint32_t*>(&h[0]);
  mid = *reinterpret_cast<const uint32_t*>(&h[1]);
  lo = *reinterpret_cast<const uint32_t*>(&h[2]);
}

// The activation as a constant of the code that runs over many values: a
// branch at each of them would keep their exponentials from overlapping.
template <class Fn>
__device__ __forceinline__ void with_act(int act, Fn fn) {
  if (act)
    fn(std::integral_constant<int, 1>{});
  else
    fn(std::integral_constant<int, 0>{});
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 32 bytes in one store: a whole sector of memory, which two of 16 are not.
// p on 32 bytes.
struct alignas(32) Vec32 {
  uint32_t w[8];
};
__device__ __forceinline__ void store32(__nv_bfloat16* p, const uint32_t (&w)[8]) {
  Vec32* to = HND_G(reinterpret_cast<Vec32*>(p));
#ifdef HYENA_ND_BOUNDS
  // where the check sends a stray store there is room, but 16-byte alignment
  to = reinterpret_cast<Vec32*>((reinterpret_cast<uintptr_t>(to) + 31) & ~uintptr_t{31});
#endif
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to),
               "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

__device__ __forceinline__ void stage_put(uint32_t addr, float v) {
  const __nv_bfloat16 h = __float2bfloat16_rn(v);
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(*reinterpret_cast<const uint16_t*>(&h)));
}

// ------------------------------------------------------------------- kernel
struct Tile {
  int split, batch, mt, nt;
};

// Keeps a value in its register: launch parameters picked by a running index
// are otherwise read again at each use, a dependent load of some 50 cycles,
// and the issuing warps then take longer for a stage than its products.
__device__ __forceinline__ int pinned(int v) {
  asm volatile("" : "+r"(v));
  return v;
}
__device__ __forceinline__ Div pinned(const Div& d) {
  return Div{static_cast<uint32_t>(pinned(static_cast<int>(d.d))), static_cast<uint32_t>(pinned(static_cast<int>(d.mul))),
             static_cast<uint32_t>(pinned(static_cast<int>(d.shift)))};
}

// A warp's way through the tiles: the current job's shape in registers.
// Tiles run in groups of eight m tiles over all n tiles, so that the tiles in
// flight share both operands in L2.
struct Walk {
  int job = -1, begin = 0, end = 0;
  int mm, mt, splits, stages, kper;
  Div per, group8, mdiv;

  __device__ __forceinline__ void seek(const Params& p, int t) {      // t never falls
    while (t >= end) {
      const Job& j = p.job[++job];
      mt = pinned(j.mt);
      mm = pinned(j.batches * j.mt);
      splits = pinned(j.splits);
      stages = pinned(j.kbatches * j.kblocks);
      kper = pinned(j.kper);
      per = pinned(j.per), group8 = pinned(j.group8), mdiv = pinned(j.mdiv);
      begin = end;
      end += static_cast<int>(per.d) * splits;
    }
  }
  __device__ __forceinline__ int split(int t) const { return splits > 1 ? per.quot(t - begin) : 0; }
  __device__ __forceinline__ Tile tile(int t) const {
    Tile r{};
    r.split = split(t);
    t -= begin + r.split * static_cast<int>(per.d);
    const int g = group8.quot(t), rows = min(8, mm - 8 * g);
    t -= g * static_cast<int>(group8.d);
    r.nt = rows == 8 ? t >> 3 : t / rows;
    const int m = 8 * g + t - r.nt * rows;
    r.batch = mdiv.quot(m);
    r.mt = m - r.batch * mt;
    return r;
  }
  // The stages [lo, hi) of a split, and how many pieces of PIECE they are.
  __device__ __forceinline__ void range(int split, int& lo, int& hi) const {
    lo = min(stages, split * kper);
    hi = min(stages, lo + kper);
  }
};
template <bool F32>
__device__ __forceinline__ int pieces_of(const Params& p, int lo, int hi) {
  return F32 ? (hi - lo + p.piece - 1) / p.piece : 1;
}

// Waits with the whole warp: all lanes go on or none.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int* status) {
  return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity, status));
}

// Plane products of fp32 operands, the smallest first.
__device__ __forceinline__ void planes_of(int combo, int& a, int& b) {
  a = (0x201100 >> (4 * (5 - combo))) & 0xF;   // low high, high low, mid mid, mid high, high mid, high high
  b = (0x021010 >> (4 * (5 - combo))) & 0xF;
}

template <int EPI, bool F32>
struct Plan {
  static constexpr int kTurns = EPI == kEpiGrad && !F32 ? 2 : 1;    // of G and U in a tile
  static constexpr int kSegs = kTurns + 1;                          // segments of a job at most
  static constexpr bool kSums = F32 && EPI != kEpiGrad;             // pieces add up in the other accumulator
  static constexpr int kBufs = kTurns == 2 || kSums ? 1 : 2;        // accumulators of 256 columns
  // columns of a tile: hidden channels, or columns of D.  The fp32 gradients
  // have fewer: a thread holds its columns' sums in registers
  static constexpr int kCols = EPI == kEpiHidden ? 128 : F32 && EPI == kEpiGrad ? 64 : 256;
  static constexpr int kOuts = EPI == kEpiGrad ? 3 : 1;
  // Four warps of epilogue see all lanes; two such groups share the columns,
  // or four where little else runs under them (bf16 gradients).
  static constexpr int kGroups = EPI == kEpiGrad && !F32 ? 4 : 2;
  static constexpr int kThreads = 32 * (3 + 4 * kGroups);           // a warp for A's copies, one for the MMAs, one for B's
  // bf16 leaves by TMA, gathered in shared memory: of each group and output
  // 128 positions x kWide hidden channels, or (kEpiOut) 32 n x 128 m; where
  // there is room twice, so that a copy out runs under the next gathering
  static constexpr int kWide = EPI == kEpiGrad ? 32 : 64;
  static constexpr int kStoreBytes = EPI == kEpiOut ? 8192 : 256 * kWide;
  static constexpr int kStoreBufs = EPI == kEpiGrad ? 1 : 2;
  static constexpr int kGroupStore = F32 ? 0 : kStoreBufs * kOuts * kStoreBytes;
  static constexpr int kStages = F32 ? 7 : EPI == kEpiGrad ? 4 : EPI == kEpiHidden ? 5 : 6;
  static constexpr int kSmem = 1024 + kStages * kStage + kGroups * kGroupStore + 8 * (2 * kStages + 2 * kBufs) + 16;
};

template <int EPI, bool F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Plan<EPI, F32>::kThreads, 1)
    k_ffn_gemm(const __grid_constant__ Params p) {
  using PL = Plan<EPI, F32>;
  extern __shared__ __align__(16) unsigned char hnd_dyn_smem[];
  const uint32_t base = (s32(hnd_dyn_smem) + 1023) & ~1023u;
  const uint32_t out = base + PL::kStages * kStage;
  const uint32_t bars = out + PL::kGroups * PL::kGroupStore;
  const uint32_t full = bars, empty = full + 8 * PL::kStages, accf = empty + 8 * PL::kStages,
                 acce = accf + 8 * PL::kBufs, tmem_slot = acce + 8 * PL::kBufs;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_rank();
  const int pairs = gridDim.x / 2, pair = blockIdx.x / 2;
  const int combos = F32 ? 6 : 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < PL::kStages; ++i) bar_init(full + 8 * i, 1), bar_init(empty + 8 * i, 1);
    for (int i = 0; i < PL::kBufs; ++i) bar_init(accf + 8 * i, 1), bar_init(acce + 8 * i, 8 * PL::kGroups);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tmem_slot) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  tmem_fence_before();
  __syncthreads();
  cluster_sync();
  tmem_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot));
  // so far under the kernel in front; the next one may set itself up too
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  bool ok = true;
  if (warp == 0 || warp == PL::kThreads / 32 - 1) {
    // ---- TMA: this CTA's 128 rows of A (first warp) and its part of B (last
    // warp).  A warp goes through the loop as one and a single lane issues:
    // under a branch on the lane every operand of a copy would first have to
    // be made uniform.
    const bool lead = elected(), is_b = warp != 0;
    int st = 0, ph = 0;
    const uint32_t lead_full = in_leader(full);
    Walk walk;
    constexpr int S = PL::kSegs;
    int job = -1, nseg = 0, kblocks = 0, wide = 0, mn[S], half_n[S], step[S], off[S], batched[S];
    uint32_t bytes[S];
    const CUtensorMap* map[S];
    bool long_k = false;
    for (int t = pair; ok && t < p.tiles; t += pairs) {
      walk.seek(p, t);
      if (walk.job != job) {
        job = walk.job;
        const Job& j = p.job[job];
        nseg = pinned(j.nseg);
        kblocks = pinned(j.kblocks);
        long_k = pinned(j.kbatches) > 1;
        wide = pinned(static_cast<int>(j.N));
#pragma unroll
        for (int i = 0; i < S; ++i) {
          const Seg& s = p.seg[j.seg0 + (i < nseg ? i : 0)];
          mn[i] = pinned(is_b ? s.b_mn : s.a_mn);
          half_n[i] = pinned(is_b ? s.ncols / 2 : 128);
          step[i] = pinned(is_b ? s.nstep : 256);
          off[i] = pinned(static_cast<int>(rank) * (is_b ? s.noff : 128) + (is_b ? s.nbase : 0));
          batched[i] = pinned(is_b ? s.b_batched : s.a_batched);
          // MN-major boxes are 64 wide, also where fewer are used
          bytes[i] = pinned(2 * (kHalf + 2 * kBK * (s.b_mn && s.ncols < 128 ? 64 : s.ncols / 2)));
          map[i] = &p.map[pinned(is_b ? (rank ? s.b1 : s.b0) : s.a)];
        }
      }
      const Tile ti = walk.tile(t);
      int lo, hi;
      walk.range(ti.split, lo, hi);
      const int pieces = pieces_of<F32>(p, lo, hi);
      for (int pc = 0; ok && pc < pieces * combos; ++pc) {
        int plane = 0;
        if (F32) {
          int pa, pb;
          planes_of(pc % combos, pa, pb);
          plane = is_b ? pb * p.b_plane : pa * p.a_plane;
        }
        const int from = F32 ? lo + pc / combos * p.piece : lo, to = F32 ? min(hi, from + p.piece) : hi;
#pragma unroll
        for (int i = 0; i < S; ++i) {
          if (i >= nseg || (i == 2 && ti.nt * 256 + 128 >= wide)) continue;      // no second turn behind the last channel
          const int r0 = (is_b ? ti.nt : ti.mt) * step[i] + off[i];
          int bat = long_k ? from / kblocks : ti.batch, k = (long_k ? from - bat * kblocks : from) * kBK;
          for (int kb = from; ok && kb < to; ++kb) {
            if (!(ok = warp_wait(empty + 8 * st, ph ^ 1, p.status))) break;
            const int z = plane + (batched[i] ? bat : 0);
            const uint32_t dst = base + st * kStage + (is_b ? kHalf : 0), bar = lead_full + 8 * st;
            if (lead) {
              if (rank == 0 && !is_b) bar_expect(full + 8 * st, bytes[i]);
              if (mn[i]) {
                tma_load(dst, map[i], bar, r0, k, z);
                if (half_n[i] > 64) tma_load(dst + 8192, map[i], bar, r0 + 64, k, z);
              } else {
                tma_load(dst, map[i], bar, k, r0, z);
              }
            }
            __syncwarp();
            if (++st == PL::kStages) st = 0, ph ^= 1;
            k += kBK;
            if (long_k && k == kblocks * kBK) k = 0, ++bat;
          }
        }
      }
    }
    if (!ok) {   // copies in flight land before the shared memory goes: they take microseconds
      const uint64_t t0 = now_ns();
      while (now_ns() - t0 < 20000000ull) {
      }
    }
  } else if (warp == 1) {
    // ---- MMA: one lane of the leading CTA's warp
    const bool lead = elected();
    if (rank == 0) {
      constexpr int S = PL::kSegs;
      int st = 0, ph = 0, buf = 0, bph = 0, job = -1, nseg = 0, wide = 0, a_mn[S], b_mn[S], acc[S], clear[S];
      uint32_t id[S];
      Walk walk;
      for (int t = pair; ok && t < p.tiles; t += pairs) {
        walk.seek(p, t);
        if (walk.job != job) {
          job = walk.job;
          const Job& j = p.job[job];
          nseg = pinned(j.nseg);
          wide = pinned(static_cast<int>(j.N));
#pragma unroll
          for (int i = 0; i < S; ++i) {
            const Seg& s = p.seg[j.seg0 + (i < nseg ? i : 0)];
            a_mn[i] = pinned(s.a_mn), b_mn[i] = pinned(s.b_mn);
            acc[i] = pinned(s.acc), clear[i] = pinned(s.clear);
            id[i] = pinned(instruction(s.a_mn, s.b_mn, s.ncols));
          }
        }
        int lo, hi;
        walk.range(walk.split(t), lo, hi);
        // what is handed to the epilogue at a time: a piece of fp32's sums, or a turn of G and U
        int pieces = pieces_of<F32>(p, lo, hi);
        if (PL::kTurns == 2) pieces = walk.tile(t).nt * 256 + 128 < wide ? 2 : 1;
        for (int pc = 0; ok && pc < pieces; ++pc) {
          if (!(ok = warp_wait(acce + 8 * buf, bph ^ 1, p.status))) break;
          tmem_fence_after();
          const int from = F32 ? lo + pc * p.piece : lo, to = F32 ? min(hi, from + p.piece) : hi;
          for (int c = 0; ok && c < combos; ++c)
#pragma unroll
            for (int i = 0; i < S; ++i) {
              if (i >= nseg || (PL::kTurns == 2 && (i == 2) != (pc == 1))) continue;
              const uint32_t d = tmem + buf * 256 + acc[i];
              const uint32_t da = a_mn[i] ? 2048 >> 4 : 32 >> 4, db = b_mn[i] ? 2048 >> 4 : 32 >> 4;
              bool add = c > 0 || !clear[i];
              for (int kb = from; ok && kb < to; ++kb) {
                if (!(ok = warp_wait(full + 8 * st, ph, p.status))) break;
                tmem_fence_after();
                const uint32_t sa = base + st * kStage;
                const uint64_t a = operand(sa, a_mn[i]), b = operand(sa + kHalf, b_mn[i]);
                if (lead) {
#pragma unroll
                  for (int q = 0; q < kBK / 16; ++q) mma(d, a + q * da, b + q * db, id[i], add || q > 0);
                  mma_commit(empty + 8 * st);
                }
                __syncwarp();
                add = true;
                if (++st == PL::kStages) st = 0, ph ^= 1;
              }
            }
          if (lead) mma_commit(accf + 8 * buf);
          __syncwarp();
          if (++buf == PL::kBufs) buf = 0, bph ^= 1;
        }
      }
    }
  } else {
    // ---- epilogue: groups of four warps, each takes its part of the columns
    constexpr int GR = PL::kGroups;
    const int quad = warp % 4, group = (warp - 2) / 4, row = quad * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const bool issuer = (warp - 2) % 4 == 0 && lane == 0;
    const uint32_t stage = out + group * PL::kGroupStore;
    int buf = 0, bph = 0, sbuf = 0;
    // all four warps of the group go on, or none: they meet at barriers below
    auto arrived = [&] {
      const bool yes = named_all(1 + group, 128, bar_wait(accf + 8 * buf, bph, p.status));
      tmem_fence_after();
      return yes;
    };
    auto release = [&] {
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_cluster(in_leader(acce + 8 * buf));
      if (++buf == PL::kBufs) buf = 0, bph ^= 1;
    };
    Walk walk;
    for (int t = pair; t < p.tiles; t += pairs) {
      walk.seek(p, t);
      const Tile ti = walk.tile(t);
      const Job& j = p.job[walk.job];
      const int m0 = ti.mt * 256 + static_cast<int>(rank) * 128;
      const long long m = m0 + row;
      const bool live = m < j.M;
      if constexpr (PL::kSums) {
        int lo, hi;
        walk.range(ti.split, lo, hi);
        const int pieces = pieces_of<F32>(p, lo, hi);
        const uint32_t acc = tmem + lanes;
        // columns from c on, 32 of them: the last piece's on the sum of those before
        auto gather = [&](uint32_t (&v)[32], int c, bool more) {
          tmem_load(v, acc + c);
          if (more) {
            uint32_t before[32];
            tmem_load(before, acc + 256 + c);
            tmem_wait_load();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(before[i]));
          } else {
            tmem_wait_load();
          }
        };
        // the columns of this group: of each product, half of a tile's
        constexpr int Q = EPI == kEpiOut ? 1 : 2;
        const int cols = EPI == kEpiOut ? pinned(j.cols) : PL::kCols, per = cols / GR;
        bool yes = true;
        for (int pc = 0; pc < pieces - 1 && (yes = arrived()); ++pc) {
#pragma unroll 1
          for (int c = 0; c < Q * per; c += 32) {
            const int col = c / per * PL::kCols + group * per + c % per;
            if (ti.nt * cols + group * per + c % per >= j.N) continue;      // no such columns
            uint32_t v[32];
            gather(v, col, pc > 0);
            tmem_store(acc + 256 + col, v);
          }
          tmem_wait_store();
          release();
        }
        if (!yes || !arrived()) break;
        const bool more = pieces > 1;
        if constexpr (EPI == kEpiOut) {
          const long long at = j.group > 0 ? (m / j.group) * j.gs + m % j.group : m;
#pragma unroll 1
          for (int c = 0; c < per; c += 32) {
            const int n0 = ti.nt * cols + group * per + c;
            uint32_t v[32];
            if (n0 < j.N) gather(v, group * per + c, more);
            if (c + 32 == per) release();
            if (n0 >= j.N) continue;
            if (j.kind == kOutF32) {
              float* o = static_cast<float*>(j.ptr) + (static_cast<long long>(ti.split) * j.batches + ti.batch) * j.bs + at;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (live && n0 + i < j.N) *HND_G(o + (n0 + i) * j.rs) = __uint_as_float(v[i]);
            } else {
              // token-major: a lane's columns are adjacent (N is a multiple of 8)
              float* o = static_cast<float*>(j.ptr) + m * j.rs + n0;
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                if (live && n0 + i < j.N)
                  *HND_G(reinterpret_cast<uint4*>(o + i)) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < per; c += 32) {
            const int n0 = ti.nt * cols + group * per + c;
            uint32_t g[32], u[32];
            if (n0 < j.N) {
              gather(g, group * per + c, more);
              gather(u, PL::kCols + group * per + c, more);
            }
            if (c + 32 == per) release();
            if (n0 >= j.N) continue;
            __nv_bfloat16* o = p.hid[0] + m * p.hid_rs + n0;
            with_act(p.act, [&](auto kind) {
              constexpr int ACT = decltype(kind)::value;
#pragma unroll
              for (int i0 = 0; i0 < 32; i0 += 16) {
                uint32_t w[3][8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const int at = i0 + 2 * i;
                  const float gv[2] = {__uint_as_float(g[at]), __uint_as_float(g[at + 1])};
                  const float uv[2] = {__uint_as_float(u[at]), __uint_as_float(u[at + 1])};
                  float h[2];
                  hidden2<true, ACT>(gv, uv, h);
                  split3x2(h[0], h[1], w[0][i], w[1][i], w[2][i]);
                }
                if (live && n0 + i0 < j.N)
#pragma unroll
                  for (int k = 0; k < 3; ++k) store32(o + k * p.hid_plane + i0, w[k]);
              }
            });
          }
        }
      } else if constexpr (F32) {
        // sum[q][i]: product q of the tile at this group's column i
        constexpr int W = PL::kCols / GR;
        float sum[3][W];
        int lo, hi;
        walk.range(ti.split, lo, hi);
        const int pieces = pieces_of<F32>(p, lo, hi);
        bool yes = true;
        for (int pc = 0; pc < pieces; ++pc) {
          if (!(yes = arrived())) break;
          const uint32_t acc = tmem + lanes + buf * 256 + group * W;
#pragma unroll
          for (int q = 0; q < 3; ++q)
#pragma unroll
            for (int c0 = 0; c0 < W; c0 += 32) {
              uint32_t v[32];
              tmem_load(v, acc + q * PL::kCols + c0);
              tmem_wait_load();
#pragma unroll
              for (int i = 0; i < 32; ++i)
                sum[q][c0 + i] = pc ? sum[q][c0 + i] + __uint_as_float(v[i]) : __uint_as_float(v[i]);
            }
          release();
        }
        if (!yes) break;
        const int n0 = ti.nt * PL::kCols + group * W;
        __nv_bfloat16* o = p.hid[0] + m * p.hid_rs + n0;
        const long long apart[3] = {0, p.hid[1] - p.hid[0], p.hid[2] - p.hid[0]};
        with_act(p.act, [&](auto kind) {
          constexpr int ACT = decltype(kind)::value;
#pragma unroll
          for (int i = 0; i < W; i += 2) {      // the hidden values take the place of the sums
            const float g[2] = {sum[0][i], sum[0][i + 1]}, u[2] = {sum[1][i], sum[1][i + 1]};
            const float d[2] = {sum[2][i], sum[2][i + 1]};
            float r[3][2];
            hidden_grads2<true, ACT>(g, u, d, r[0], r[1], r[2]);
#pragma unroll
            for (int q = 0; q < 3; ++q) sum[q][i] = r[q][0], sum[q][i + 1] = r[q][1];
          }
        });
#pragma unroll
        for (int q = 0; q < 3; ++q)
#pragma unroll
          for (int i0 = 0; i0 < W; i0 += 16) {
            uint32_t w[3][8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              split3x2(sum[q][i0 + 2 * i], sum[q][i0 + 2 * i + 1], w[0][i], w[1][i], w[2][i]);
            if (live && n0 + i0 < j.N)
#pragma unroll
              for (int k = 0; k < 3; ++k) store32(o + apart[q] + k * p.hid_plane + i0, w[k]);
          }
      } else {
        if constexpr (EPI == kEpiOut) {
          if (!arrived()) break;
          const int per = pinned(j.cols) / GR;
          const uint32_t acc = tmem + lanes + buf * 256 + group * per;
          const long long at = j.group > 0 ? (m / j.group) * j.gs + m % j.group : m;
          for (int c0 = 0; c0 < per; c0 += 32) {
            const int n0 = ti.nt * per * GR + group * per + c0;
            uint32_t v[32];
            if (n0 < j.N) {      // such columns exist
              tmem_load(v, acc + c0);
              tmem_wait_load();
            }
            if (c0 + 32 == per) release();
            if (n0 >= j.N) continue;
            if (j.kind == kOutTma) {
              const uint32_t sb = stage + sbuf * PL::kStoreBytes;
              if (issuer) store_wait_read<1>();
              named_sync(1 + group, 128);
#pragma unroll
              for (int i = 0; i < 32; ++i) stage_put(sb + i * 256 + row * 2, __uint_as_float(v[i]));
              fence_async();
              named_sync(1 + group, 128);
              if (issuer && m0 < j.M && n0 < j.N) tma_store(&p.map[j.map], sb, m0, n0, ti.batch);
              if (issuer) store_commit();
              sbuf ^= 1;
            } else if (j.kind == kOutBf16) {
              __nv_bfloat16* o = static_cast<__nv_bfloat16*>(j.ptr) + at;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (live && n0 + i < j.N) *HND_G(o + (n0 + i) * j.rs) = __float2bfloat16_rn(__uint_as_float(v[i]));
            } else if (j.kind == kOutF32) {
              float* o = static_cast<float*>(j.ptr) + (static_cast<long long>(ti.split) * j.batches + ti.batch) * j.bs + m;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (live && n0 + i < j.N) *HND_G(o + (n0 + i) * j.rs) = __uint_as_float(v[i]);
            } else {
              // token-major: a lane's columns are adjacent (N is a multiple of 8)
              __nv_bfloat16* o = static_cast<__nv_bfloat16*>(j.ptr) + m * j.rs + n0;
#pragma unroll
              for (int i = 0; i < 32; i += 8)
                if (live && n0 + i < j.N) {
                  uint32_t w[4];
#pragma unroll
                  for (int q = 0; q < 4; ++q) w[q] = pack2(__uint_as_float(v[i + 2 * q]), __uint_as_float(v[i + 2 * q + 1]));
                  *HND_G(reinterpret_cast<uint4*>(o + i)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
          }
        } else {
          // a turn's 128 hidden channels: 64 or 32 of each group, 16 at a time, gathered as rows of kWide channels of a
          // position (a thread's own 32-byte stores leave an SM at 16 bytes a cycle: 90 us for the gradients at C
          // 256, F 1024, 32768 positions)
          constexpr int W = 16, kPer = PL::kWide / W, kChunks = PL::kWide / 8, kMine = 128 / GR;
          constexpr int kAhead = GR == 2 ? 1 : 0;      // four groups hide their latencies by turns, and have no registers
          bool yes = true;
          for (int turn = 0; turn < PL::kTurns; ++turn) {
            const int n0 = ti.nt * PL::kCols + turn * 128;
            if (n0 >= j.N || !(yes = arrived())) break;
            const uint32_t acc = tmem + lanes + buf * 256 + group * kMine;
            // the next 16 channels are on their way while these are worked on
            uint32_t g[kAhead + 1][W], u[kAhead + 1][W], d[kAhead + 1][EPI == kEpiGrad ? W : 1];
            auto load = [&](int c) {
              tmem_load(g[c & kAhead], acc + c * W);
              tmem_load(u[c & kAhead], acc + 128 + c * W);
              if constexpr (EPI == kEpiGrad) tmem_load(d[c & kAhead], acc + 256 + turn * 128 + c * W);
            };
            load(0);
            with_act(p.act, [&](auto kind) {
              constexpr int ACT = decltype(kind)::value;
#pragma unroll
              for (int c = 0; c < kMine / W; ++c) {
                if (!kAhead && c) load(c);
                tmem_wait_load();
                if (kAhead && c + 1 < kMine / W) load(c + 1);
                if (c + 1 == kMine / W) release();
                const uint32_t to = stage + sbuf * (PL::kOuts * PL::kStoreBytes);
                if (c % kPer == 0) {      // this buffer's copies before the last have left it
                  if (issuer) store_wait_read<PL::kStoreBufs - 1>();
                  named_sync(1 + group, 128);
                }
                uint32_t w[PL::kOuts][8];
#pragma unroll
                for (int i = 0; i < W; i += 2) {
                  const float gv[2] = {__uint_as_float(g[c & kAhead][i]), __uint_as_float(g[c & kAhead][i + 1])};
                  const float uv[2] = {__uint_as_float(u[c & kAhead][i]), __uint_as_float(u[c & kAhead][i + 1])};
                  float r[3][2];
                  if constexpr (EPI == kEpiGrad) {
                    const float dv[2] = {__uint_as_float(d[c & kAhead][i]), __uint_as_float(d[c & kAhead][i + 1])};
                    hidden_grads2<false, ACT>(gv, uv, dv, r[0], r[1], r[2]);
                  } else {
                    hidden2<false, ACT>(gv, uv, r[0]);
                  }
#pragma unroll
                  for (int q = 0; q < PL::kOuts; ++q) w[q][i / 2] = pack2(r[q][0], r[q][1]);
                }
                // 16-byte chunks of the row, under the 64- or 128-byte swizzle
                const int key = kChunks == 8 ? row & 7 : row >> 1 & 3;
#pragma unroll
                for (int q = 0; q < PL::kOuts; ++q)
#pragma unroll
                  for (int i = 0; i < 2; ++i)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     to + q * PL::kStoreBytes + row * (2 * PL::kWide) +
                                     (((c % kPer * 2 + i) ^ key) << 4)),
                                 "r"(w[q][4 * i]), "r"(w[q][4 * i + 1]), "r"(w[q][4 * i + 2]), "r"(w[q][4 * i + 3])
                                 : "memory");
                if (c % kPer == kPer - 1) {
                  fence_async();
                  named_sync(1 + group, 128);
                  if (issuer) {
                    const int n = n0 + group * kMine + c / kPer * PL::kWide;
                    if (m0 < j.M && n < j.N)
#pragma unroll
                      for (int q = 0; q < PL::kOuts; ++q)
                        tma_store(&p.map[p.hmap[q]], to + q * PL::kStoreBytes, n, m0, ti.batch);
                    store_commit();
                  }
                  sbuf = (sbuf + 1) % PL::kStoreBufs;
                }
              }
            });
          }
          if (!yes) break;
        }
      }
    }
    if (!F32 && issuer) store_wait_read<0>();
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

}  // namespace ffn
}  // namespace hnd
