// The residual join with the norms on both sides of it, forward and backward.
#include "hnd_join.cuh"

namespace hnd {

// ----------------------------------------- any number of channels, any length
// For more channels than a block of hnd_join.cuh holds in registers: a block
// takes 32 positions and reads their channels again for each of its sweeps,
// from L2 mostly.  Such a block holds (join_plan), with rows of whole 16-byte
// vectors, 16384 channels of a token forward and 8192 in the gradients, of a
// grid's positions 4096 (fp32) or 2048 (bf16) forward and 2048 in the
// gradients; with other rows 8192 and 4096 of a token, 16384 and 4096 of a
// grid.
constexpr int kJoinLanes = 32;   // positions of a block
constexpr int kJoinRows = 8;     // channel rows of a block

// One position's view of the join: values at channel c.
template <class TT>
struct Pos {
  const JoinDev& j;
  const TT *x, *y;
  long long b, base;      // sample, index of channel 0 in [B, C, L]
  DropState ds;
  float mu1 = 0.f, rho1 = 1.f, mu2 = 0.f, rho2 = 1.f;

  __device__ Pos(const JoinDev& jj, const TT* xx, const TT* yy, long long t) : j(jj), x(xx), y(yy), ds{} {
    b = t / j.L;
    base = b * j.C * j.L + t % j.L;
    if (j.border) ds = drop_state(j.rng);
  }
  __device__ long long at(long long c) const { return base + c * j.L; }
  __device__ float yhat(long long c) const { return (ld1(y + at(c)) - mu1) * rho1; }
  __device__ float w1(long long c) const { return j.w1 ? ld1(j.w1 + c) : 1.f; }
  __device__ float w2(long long c) const { return j.w2 ? ld1(j.w2 + c) : 1.f; }
  __device__ float m(long long c) const {
    if (!j.border) return 1.f;
    const long long i = at(c);
    return drop_lot(drop_lots(ds, static_cast<uint64_t>(i >> 3)), static_cast<int>(i & 7)) >= j.border ? j.factor
                                                                                                       : 0.f;
  }
  __device__ float sg(long long c) const {
    return (j.scale ? ld1(j.scale + c) : 1.f) * (j.gate ? ld1(j.gate + b * j.C + c) : 1.f);
  }
  __device__ float h(long long c) const {
    const float xv = ld1(x + at(c));
    if (!y) return xv;
    const float f = m(c);
    if (f == 0.f) return xv;
    const float z = yhat(c) * w1(c) + (j.b1 ? ld1(j.b1 + c) : 0.f);
    return xv + sg(c) * (f * z);
  }
  __device__ float hhat(long long c) const { return (h(c) - mu2) * rho2; }
};

// Sum over the channel rows of a block, for each of its positions.
__device__ __forceinline__ float rows_sum(float v, float (*buf)[kJoinLanes]) {
  __syncthreads();
  buf[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int r = 0; r < kJoinRows; ++r) s += buf[r][threadIdx.x];
  return s;
}

// Mean and reciprocal deviation of f(c) over the channels.
template <class Fn>
__device__ __forceinline__ void norm_stats(int kind, float eps, long long C, bool live, float (*buf)[kJoinLanes],
                                           float& mu, float& rho, Fn f) {
  mu = 0.f;
  rho = 1.f;
  if (!kind) return;
  const float inv = 1.f / static_cast<float>(C);
  if (kind == 2) {
    float s = 0.f;
    if (live)
      for (long long c = threadIdx.y; c < C; c += kJoinRows) s += f(c);
    mu = rows_sum(s, buf) * inv;
  }
  float s = 0.f;
  if (live)
    for (long long c = threadIdx.y; c < C; c += kJoinRows) {
      const float d = f(c) - mu;
      s += d * d;
    }
  rho = rsqrtf(rows_sum(s, buf) * inv + eps);
}

template <class TT>
__device__ __forceinline__ void pos_stats(Pos<TT>& p, bool live, float (*buf)[kJoinLanes]) {
  const JoinDev& j = p.j;
  if (p.y) {
    float mu, rho;
    norm_stats(j.post, j.eps1, j.C, live, buf, mu, rho, [&](long long c) { return ld1(p.y + p.at(c)); });
    p.mu1 = mu;
    p.rho1 = rho;
  }
  float mu, rho;
  norm_stats(j.pre, j.eps2, j.C, live, buf, mu, rho, [&](long long c) { return p.h(c); });
  p.mu2 = mu;
  p.rho2 = rho;
}

template <class TT>
__global__ void __launch_bounds__(kJoinLanes* kJoinRows)
    k_join_any_fwd(JoinDev j, const TT* __restrict__ x, const TT* __restrict__ y, TT* __restrict__ h, TT* __restrict__ n) {
  __shared__ float buf[kJoinRows][kJoinLanes];
  const long long t = blockIdx.x * static_cast<long long>(kJoinLanes) + threadIdx.x;
  const bool live = t < j.T;
  Pos<TT> p(j, x, y, live ? t : 0);
  pos_stats(p, live, buf);
  if (!live) return;
  for (long long c = threadIdx.y; c < j.C; c += kJoinRows) {
    const float hv = p.h(c);
    if (h) st1(h + p.at(c), hv);
    if (n) st1(n + p.at(c), (hv - p.mu2) * p.rho2 * p.w2(c) + (j.b2 ? ld1(j.b2 + c) : 0.f));
  }
}

// Statistics of a position that the parameter gradients need again.
struct JoinStat {
  float mu1, rho1, mu2, rho2, s1, s2, pad0, pad1;
};

template <class TT>
__device__ __forceinline__ float whole_grad(const Pos<TT>& p, const TT* dh, const TT* dn, long long c, float s1,
                                            float s2) {
  float d = dh ? ld1(dh + p.at(c)) : 0.f;
  if (dn) d += p.rho2 * (ld1(dn + p.at(c)) * p.w2(c) - s1 - p.hhat(c) * s2);
  return d;
}

template <class TT>
__global__ void __launch_bounds__(kJoinLanes* kJoinRows)
    k_join_any_bwd(JoinDev j, const TT* __restrict__ x, const TT* __restrict__ y, const TT* __restrict__ dh,
               const TT* __restrict__ dn, TT* __restrict__ dx, TT* __restrict__ dy, JoinStat* __restrict__ stats) {
  __shared__ float buf[kJoinRows][kJoinLanes];
  const long long t = blockIdx.x * static_cast<long long>(kJoinLanes) + threadIdx.x;
  const bool live = t < j.T;
  Pos<TT> p(j, x, y, live ? t : 0);
  pos_stats(p, live, buf);
  const float inv = 1.f / static_cast<float>(j.C);
  float s1 = 0.f, s2 = 0.f;
  if (dn && live)
    for (long long c = threadIdx.y; c < j.C; c += kJoinRows) {
      const float a = ld1(dn + p.at(c)) * p.w2(c);
      s1 += a;
      s2 += a * p.hhat(c);
    }
  s1 = j.pre == 2 ? rows_sum(s1, buf) * inv : 0.f;
  s2 = rows_sum(s2, buf) * inv;
  float s3 = 0.f, s4 = 0.f;
  if (y && j.post) {
    if (live)
      for (long long c = threadIdx.y; c < j.C; c += kJoinRows) {
        const float f = p.m(c);
        if (f == 0.f) continue;
        const float e = whole_grad(p, dh, dn, c, s1, s2) * f * p.sg(c) * p.w1(c);
        s3 += e;
        s4 += e * p.yhat(c);
      }
    s3 = j.post == 2 ? rows_sum(s3, buf) * inv : 0.f;
    s4 = rows_sum(s4, buf) * inv;
  }
  if (!live) return;
  for (long long c = threadIdx.y; c < j.C; c += kJoinRows) {
    const float d = whole_grad(p, dh, dn, c, s1, s2);
    st1(dx + p.at(c), d);
    if (y) {
      const float f = p.m(c);
      const float e = f == 0.f ? 0.f : d * f * p.sg(c) * p.w1(c);
      st1(dy + p.at(c), j.post ? p.rho1 * (e - s3 - p.yhat(c) * s4) : e);
    }
  }
  if (threadIdx.y == 0) *HND_G(stats + t) = JoinStat{p.mu1, p.rho1, p.mu2, p.rho2, s1, s2, 0.f, 0.f};
}

// Per (b, c): sums over the positions of dht m yhat, dht m, dn hhat, dn.
template <class TT>
__global__ void __launch_bounds__(256)
    k_join_any_param(JoinDev j, const TT* __restrict__ x, const TT* __restrict__ y, const TT* __restrict__ dh,
                 const TT* __restrict__ dn, const JoinStat* __restrict__ stats, float4* __restrict__ part) {
  const long long bc = blockIdx.x, b = bc / j.C, c = bc % j.C;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (long long l = threadIdx.x; l < j.L; l += 256) {
    const long long t = b * j.L + l;
    Pos<TT> p(j, x, y, t);
    const JoinStat st = *HND_G(stats + t);
    p.mu1 = st.mu1, p.rho1 = st.rho1, p.mu2 = st.mu2, p.rho2 = st.rho2;
    if (y) {
      const float f = p.m(c);
      if (f != 0.f) {
        const float d = whole_grad(p, dh, dn, c, st.s1, st.s2) * f;
        s.x += d * p.yhat(c);
        s.y += d;
      }
    }
    if (dn) {
      const float v = ld1(dn + p.at(c));
      s.z += v * p.hhat(c);
      s.w += v;
    }
  }
  __shared__ float4 buf[256];
  buf[threadIdx.x] = s;
  __syncthreads();
  for (int k = 128; k > 0; k /= 2) {
    if (threadIdx.x < k) {
      float4 &u = buf[threadIdx.x], v = buf[threadIdx.x + k];
      u.x += v.x, u.y += v.y, u.z += v.z, u.w += v.w;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) *HND_G(part + bc) = buf[0];
}

// ------------------------------------------------- gradients of parameters
struct JoinGradsDev {
  float *w1, *b1, *gate, *scale, *w2, *b2;
};

// The parameters' gradients from the blocks' sums, `per` rows a sample (0:
// already weighted with the gate).  The first ceil(C / 32) blocks sum over
// all rows, the next over those of sample 0 for its gate, and so on.
__global__ void __launch_bounds__(1024)
    k_join_grads(const JoinDev j, const float4* __restrict__ part, long long rows, long long per, JoinGradsDev g) {
  __shared__ float buf[4][32][33];
  const unsigned wide = static_cast<unsigned>((j.C + 31) / 32);
  const long long c = blockIdx.x % wide * 32LL + threadIdx.x, gate_of = static_cast<long long>(blockIdx.x / wide) - 1;
  const bool live = c < j.C;
  const long long lo = gate_of < 0 ? 0 : gate_of * per, hi = gate_of < 0 ? rows : lo + per;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live)
    for (long long r = lo + threadIdx.y; r < hi; r += 32) {
      const float4 v = *HND_G(part + r * j.C + c);
      const float gt = gate_of < 0 && per && j.gate ? __ldg(HND_G(j.gate + r / per * j.C + c)) : 1.f;
      s.x += gt * v.x, s.y += gt * v.y, s.z += v.z, s.w += v.w;
    }
  buf[0][threadIdx.y][threadIdx.x] = s.x;
  buf[1][threadIdx.y][threadIdx.x] = s.y;
  buf[2][threadIdx.y][threadIdx.x] = s.z;
  buf[3][threadIdx.y][threadIdx.x] = s.w;
  __syncthreads();
  // warp q of the first four adds up value q
  if (threadIdx.y < 4) {
    float v = 0.f;
    for (int r = 0; r < 32; ++r) v += buf[threadIdx.y][r][threadIdx.x];
    __syncwarp();
    buf[threadIdx.y][0][threadIdx.x] = v;
  }
  __syncthreads();
  if (threadIdx.y || !live) return;
  const float q = buf[0][0][threadIdx.x], r = buf[1][0][threadIdx.x];
  const float w1 = j.w1 ? ld1(j.w1 + c) : 1.f, b1 = j.b1 ? ld1(j.b1 + c) : 0.f, sc = j.scale ? ld1(j.scale + c) : 1.f;
  const float z = w1 * q + b1 * r;
  if (gate_of >= 0) {
    st1(g.gate + gate_of * j.C + c, sc * z);
    return;
  }
  if (g.w1) st1(g.w1 + c, sc * q);
  if (g.b1) st1(g.b1 + c, sc * r);
  if (g.scale) st1(g.scale + c, z);
  if (g.w2) st1(g.w2 + c, buf[2][0][threadIdx.x]);
  if (g.b2) st1(g.b2 + c, buf[3][0][threadIdx.x]);
}

static JoinDev device_view(const JoinArgs& a) {
  return {a.B,      a.C,      a.L,    a.B * a.L, a.post.kind, a.pre.kind,    a.post.eps,    a.pre.eps, a.post.w,
          a.post.b, a.pre.w,  a.pre.b, a.gate,    a.scale,     a.drop.border, a.drop.factor, a.drop.rng};
}

// ------------------------------------------------------------------ launches
static long long cdiv(long long a, long long b) { return (a + b - 1) / b; }

// How a call runs; a function of the shape alone.
struct JoinPlan {
  bool fast = false;       // hnd_join.cuh; else the kernels above
  bool ahead = false;      // hnd_join_grid.cuh
  int V = 1, K = 1;        // values of a vector, vectors of a thread
  int lanes = 0;           // grid: neighbouring vectors of positions; token: threads of a position
  int threads = 0;
  long long blocks = 0;
  int chunks = 1;          // gradients on grids: blocks of a sample
  long long rows = 0;      // gradients: rows of partial sums
};

constexpr long long kJoinParts = 592;     // blocks of a gradient call: four an SM

// Grid layout: the widest row of positions whose channels fit a block.
static bool grid_plan(JoinPlan& p, long long C, long long units, int widest) {
  const long long rows = cdiv(C, p.K);
  int w = widest;
  while (w > 1 && w / 2 >= units) w /= 2;
  // 256 threads, so that two blocks share an SM, unless that makes rows shorter than four vectors (32 for V = 1)
  const int least = widest / 2 < w ? widest / 2 : w;
  for (int cap : {256, kJoinMaxThreads})
    for (int v = w; v >= (cap == 256 ? least : 1); v /= 2)
      if (cdiv(v * rows, 32) * 32 <= cap) {
        p.lanes = v;
        p.threads = static_cast<int>(cdiv(v * rows, 32) * 32);
        return true;
      }
  return false;
}

// Grids of up to 512 channels (fp32 forward 1024; more where there is but one
// vector to a block): as many lanes of positions as leave threads for the channels, two
// at least where a row has two vectors.
static bool ahead_plan(JoinPlan& p, long long B, long long C, long long L, int bf16, bool backward) {
  const int V = bf16 ? 8 : 4, most = backward || bf16 ? 4 : 8;
  if (L == 1) return false;
  const bool ragged = L % V != 0;
  const long long per = cdiv(L, V), units = backward || ragged ? per : per * B;
  p.K = C <= 32 ? 1 : most;
  int w = 32;
  while (w > 1 && (256 / w * p.K < C || w / 2 >= units)) w /= 2;
  if (256 / w * p.K < C || (w == 1 && units > 1)) return false;
  p.V = V;
  p.lanes = w;
  const long long tiles = cdiv(units, w);
  if (backward) {
    // two blocks an SM: one wave of few samples, or the fullest waves of many
    const long long wave = kJoinParts / 2;
    long long chunks = B < wave ? wave / B : 1;
    for (long long c = chunks + 1; 2 * B > wave && c <= 8; ++c)
      if (c * cdiv(chunks * B, wave) > chunks * cdiv(c * B, wave)) chunks = c;
    p.chunks = static_cast<int>(tiles < chunks ? tiles : chunks);
    p.blocks = p.rows = B * p.chunks;
  } else {
    const long long all = ragged ? tiles * B : tiles;
    const long long most_blocks = ragged ? kJoinParts / 2 : 3 * kJoinParts / 4;      // two or three an SM
    p.blocks = all < most_blocks ? all : most_blocks;
  }
  p.fast = p.ahead = true;
  return true;
}

static JoinPlan join_plan(long long B, long long C, long long L, int bf16, bool backward) {
  JoinPlan p;
  if (ahead_plan(p, B, C, L, bf16, backward)) return p;
  const int wide = bf16 ? 8 : 4;
  const bool token = L == 1;
  p.V = (token ? C : L) % wide == 0 ? wide : 1;
  if (token) {
    const long long vectors = C / p.V;
    // few positions: a thread for each vector, for the shortest way through; else several, for fewer threads a row
    const int most = backward ? (p.V == 1 ? 8 : 16 / p.V) : p.V == 1 ? 16 : 32 / p.V;
    p.K = B <= 296 && vectors <= kJoinMaxThreads ? 1 : most;
    const long long t = cdiv(cdiv(vectors, p.K), 32) * 32;
    if (t > kJoinMaxThreads) return p;
    p.lanes = static_cast<int>(t);
    const long long groups = B > 296 && t < 256 ? 256 / t : 1;
    p.threads = static_cast<int>(t * groups);
    const long long tiles = cdiv(B, groups);
    p.blocks = tiles;
    if (backward) {
      const long long most_blocks = kJoinParts / groups;
      p.blocks = tiles < most_blocks ? tiles : most_blocks;
      p.rows = p.blocks * groups;
    }
  } else {
    const long long per = L / p.V, units = backward ? per : per * B;
    if (backward)
      p.K = p.V == 1 ? 8 : 4;
    else
      p.K = p.V == 1 ? 32 : 32 / wide;
    if (!grid_plan(p, C, units, p.V == 1 ? 32 : 8)) return p;
    if (backward) {
      const long long tiles = cdiv(per, p.lanes), want = cdiv(kJoinParts, B);
      p.chunks = static_cast<int>(tiles < want ? tiles : want);
      p.blocks = p.rows = B * p.chunks;
    } else {
      p.blocks = cdiv(units, p.lanes);
    }
  }
  p.fast = p.blocks < 1LL << 31;
  return p;
}

static size_t plan_smem(const JoinPlan& p, bool token) {
  const int sets = token ? 1 : p.lanes, positions = token ? 1 : p.V;
  return sizeof(float) * 2 * (p.threads / 32) * sets * 2 * positions;
}

static size_t stats_bytes(long long T) { return (static_cast<size_t>(T) * sizeof(JoinStat) + 255) / 256 * 256; }

size_t join_workspace(long long B, long long C, long long L, int bf16) {
  const JoinPlan p = join_plan(B, C, L, bf16, true);
  if (p.fast) return static_cast<size_t>(p.rows) * C * sizeof(float4);
  return stats_bytes(B * L) + static_cast<size_t>(B * C) * sizeof(float4);
}

template <class TT, int V, int K, bool TOK>
static cudaError_t forward_as(const JoinArgs& a, const JoinPlan& p) {
  k_join_fwd<TT, V, K, TOK><<<static_cast<unsigned>(p.blocks), p.threads, plan_smem(p, TOK), a.stream>>>(
      device_view(a), p.lanes, static_cast<const TT*>(a.x), static_cast<const TT*>(a.y), static_cast<TT*>(a.h),
      static_cast<TT*>(a.n));
  return cudaGetLastError();
}

template <class TT>
static cudaError_t forward(const JoinArgs& a) {
  constexpr int W = sizeof(TT) == 2 ? 8 : 4;
  const JoinPlan p = join_plan(a.B, a.C, a.L, a.bf16, false);
  if (!p.fast) {
    const JoinDev j = device_view(a);
    const unsigned blocks = static_cast<unsigned>((j.T + kJoinLanes - 1) / kJoinLanes);
    k_join_any_fwd<TT><<<blocks, dim3(kJoinLanes, kJoinRows), 0, a.stream>>>(
        j, static_cast<const TT*>(a.x), static_cast<const TT*>(a.y), static_cast<TT*>(a.h), static_cast<TT*>(a.n));
    return cudaGetLastError();
  }
  if (p.ahead) return launch_join_grid_fwd(a, device_view(a), p.lanes, p.K, static_cast<unsigned>(p.blocks));
  if (a.L == 1) {
    if (p.V == 1) return p.K == 1 ? forward_as<TT, 1, 1, true>(a, p) : forward_as<TT, 1, 16, true>(a, p);
    return p.K == 1 ? forward_as<TT, W, 1, true>(a, p) : forward_as<TT, W, 32 / W, true>(a, p);
  }
  return p.V == 1 ? forward_as<TT, 1, 32, false>(a, p) : forward_as<TT, W, 32 / W, false>(a, p);
}

// The parameters' gradients from `rows` rows of sums, `per` a sample.
static cudaError_t grads(const JoinArgs& a, const float4* part, long long rows, long long per) {
  const long long wide = cdiv(a.C, 32);
  // the checked build's table has no room for these next to the activations
  const size_t C4 = 4 * static_cast<size_t>(a.C), BC4 = C4 * static_cast<size_t>(a.B);
  BoundsList bl;
  bl.add(part, static_cast<size_t>(rows) * a.C * sizeof(float4));
  for (const float* p : {a.post.w, a.post.b, a.scale, static_cast<const float*>(a.dpost_w),
                         static_cast<const float*>(a.dpost_b), static_cast<const float*>(a.dscale),
                         static_cast<const float*>(a.dpre_w), static_cast<const float*>(a.dpre_b)})
    bl.add(p, C4);
  bl.add(a.gate, BC4);
  bl.add(a.dgate, BC4);
  const cudaError_t e = register_buffers(bl, nullptr, a.stream);
  if (e != cudaSuccess) return e;
  k_join_grads<<<static_cast<unsigned>(wide * (a.dgate && per ? 1 + a.B : 1)), dim3(32, 32), 0, a.stream>>>(
      device_view(a), part, rows, per, JoinGradsDev{a.dpost_w, a.dpost_b, a.dgate, a.dscale, a.dpre_w, a.dpre_b});
  return cudaGetLastError();
}

template <class TT, int V, int K, bool TOK>
static cudaError_t backward_as(const JoinArgs& a, const JoinPlan& p, float4* part) {
  k_join_bwd<TT, V, K, TOK><<<static_cast<unsigned>(p.blocks), p.threads, plan_smem(p, TOK), a.stream>>>(
      device_view(a), p.lanes, p.chunks, static_cast<const TT*>(a.x), static_cast<const TT*>(a.y),
      static_cast<const TT*>(a.dh), static_cast<const TT*>(a.dn), static_cast<TT*>(a.dx), static_cast<TT*>(a.dy),
      a.dgate, part);
  return cudaGetLastError();
}

template <class TT>
static cudaError_t backward(const JoinArgs& a) {
  constexpr int W = sizeof(TT) == 2 ? 8 : 4;
  const JoinPlan p = join_plan(a.B, a.C, a.L, a.bf16, true);
  const bool token = a.L == 1;
  const bool params = a.dpost_w || a.dpost_b || a.dscale || a.dpre_w || a.dpre_b || (a.dgate && !(token && p.fast));
  if (p.fast) {
    float4* part = params ? static_cast<float4*>(a.ws) : nullptr;
    cudaError_t e;
    if (p.ahead)
      e = launch_join_grid_bwd(a, device_view(a), p.lanes, p.K, p.chunks, static_cast<unsigned>(p.blocks), part);
    else if (token && p.V == 1)
      e = p.K == 1 ? backward_as<TT, 1, 1, true>(a, p, part) : backward_as<TT, 1, 8, true>(a, p, part);
    else if (token)
      e = p.K == 1 ? backward_as<TT, W, 1, true>(a, p, part) : backward_as<TT, W, 16 / W, true>(a, p, part);
    else
      e = p.V == 1 ? backward_as<TT, 1, 8, false>(a, p, part) : backward_as<TT, W, 4, false>(a, p, part);
    return e == cudaSuccess && params ? grads(a, part, p.rows, token ? 0 : p.chunks) : e;
  }
  const JoinDev j = device_view(a);
  const unsigned blocks = static_cast<unsigned>((j.T + kJoinLanes - 1) / kJoinLanes);
  JoinStat* stats = static_cast<JoinStat*>(a.ws);
  float4* part = reinterpret_cast<float4*>(static_cast<char*>(a.ws) + stats_bytes(j.T));
  const TT *x = static_cast<const TT*>(a.x), *y = static_cast<const TT*>(a.y), *dh = static_cast<const TT*>(a.dh),
           *dn = static_cast<const TT*>(a.dn);
  k_join_any_bwd<TT><<<blocks, dim3(kJoinLanes, kJoinRows), 0, a.stream>>>(j, x, y, dh, dn, static_cast<TT*>(a.dx),
                                                                          static_cast<TT*>(a.dy), stats);
  if (!params) return cudaGetLastError();
  k_join_any_param<TT><<<static_cast<unsigned>(j.B * j.C), 256, 0, a.stream>>>(j, x, y, dh, dn, stats, part);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? grads(a, part, j.B, 1) : e;
}

cudaError_t launch_join_forward(const JoinArgs& a) {
  return a.bf16 ? forward<__nv_bfloat16>(a) : forward<float>(a);
}

cudaError_t launch_join_backward(const JoinArgs& a) {
  return a.bf16 ? backward<__nv_bfloat16>(a) : backward<float>(a);
}

}  // namespace hnd
