// The gated feed-forward block over the channels of each position: operand
// layouts, the sequence of products, and the small kernels around them.
#include "hnd_block.h"
#include "hnd_ffn_few.cuh"
#include "hnd_ffn_gemm.cuh"
#include "hnd_host_util.h"
#include "hnd_io.cuh"
#include "hnd_launch.h"

namespace hnd {

using bf16 = __nv_bfloat16;
using namespace ffn;

// ------------------------------------------------------------ small kernels

// [B, C, L] -> rows c of B L adjacent positions at `pitch`: bf16 as it is,
// fp32 as three bf16 planes.  Used where samples are too short or too ragged
// for TMA, and for every fp32 operand (weights and token-major activations
// are B = 1).  All operands of a call in one launch, blockIdx.y each.
struct Pack {
  const void* x;
  bf16* out;
  long long C, L, T, pitch, plane;
};
constexpr int kMaxPacks = 5;
struct Packs {
  Pack p[kMaxPacks];
};

template <class TT>
__global__ void __launch_bounds__(256) k_ffn_pack(const Packs packs) {
  const Pack& p = packs.p[blockIdx.y];
  const TT* x = static_cast<const TT*>(p.x);
  const long long groups = p.pitch / 8, n = groups * p.C;
  for (long long g = blockIdx.x * 256LL + threadIdx.x; g < n; g += gridDim.x * 256LL) {
    const long long c = g / groups, t0 = (g - c * groups) * 8;
    long long b = t0 / p.L, l = t0 - b * p.L;
    __align__(16) bf16 v[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f = 0.f;
      if (t0 + i < p.T) f = ld1(x + (b * p.C + c) * p.L + l);
      if (++l == p.L) l = 0, ++b;
      if (sizeof(TT) == 4)
        split3(f, v[0][i], v[1][i], v[2][i]);
      else
        v[0][i] = __float2bfloat16_rn(f);
    }
#pragma unroll
    for (int k = 0; k < (sizeof(TT) == 4 ? 3 : 1); ++k)
      *HND_G(reinterpret_cast<uint4*>(p.out + k * p.plane + c * p.pitch + t0)) = *reinterpret_cast<const uint4*>(v[k]);
  }
}

// A few positions of [B, C, L] as token-major rows [plane][T][C].
template <class TT>
__global__ void __launch_bounds__(256)
    k_ffn_gather(const TT* __restrict__ x, bf16* __restrict__ out, int C, int L, int T, long long plane) {
  for (int i = blockIdx.x * 256 + threadIdx.x; i < T * C; i += gridDim.x * 256) {
    const int t = i / C, c = i % C;
    const float f = ld1(x + (static_cast<long long>(t / L) * C + c) * L + t % L);
    if constexpr (sizeof(TT) == 4) {
      bf16 v[3];
      split3(f, v[0], v[1], v[2]);
#pragma unroll
      for (int k = 0; k < 3; ++k) *HND_G(out + k * plane + i) = v[k];
    } else {
      st1(out + i, f);
    }
  }
}

// The sums of the weight gradients' partial products, in the order of the
// splits; blockIdx.y: which gradient.
struct Sums {
  void* out[3];
};

template <class TT>
__global__ void __launch_bounds__(256) k_ffn_sum(const float* __restrict__ parts, const Sums sums, long long n, int splits) {
  const float* part = parts + blockIdx.y * (n * splits);
  TT* out = static_cast<TT*>(sums.out[blockIdx.y]);
  for (long long i = (blockIdx.x * 256LL + threadIdx.x) * 4; i < n; i += gridDim.x * 1024LL) {
    float4 s = *HND_G(reinterpret_cast<const float4*>(part + i));
    for (int k = 1; k < splits; ++k) {
      const float4 v = *HND_G(reinterpret_cast<const float4*>(part + k * n + i));
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    st1(out + i, s.x), st1(out + i + 1, s.y), st1(out + i + 2, s.z), st1(out + i + 3, s.w);
  }
}

// Sums of the partial products [split][batch][C][Lx] of y or dx, back into the
// activations' layout: element (batch, c, m) of token-major positions at
// m C + c, else at (t / L) C L + c L + t % L with t the position in all.
template <class TT>
__global__ void __launch_bounds__(256)
    k_ffn_fold(const float* __restrict__ parts, TT* __restrict__ out, long long C, long long L, long long Lx, long long n,
               int splits, int token) {
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) {
    float s = 0.f;
    for (int k = 0; k < splits; ++k) s += *HND_G(parts + k * n + i);
    const long long row = i / Lx, m = i - row * Lx, b = row / C, c = row - b * C;
    if (token) {
      st1(out + m * C + c, s);
    } else {
      const long long t = b * Lx + m, sample = t / L;
      st1(out + (sample * C + c) * L + (t - sample * L), s);
    }
  }
}

// ----------------------------------------------------------------- planning
static long long up(long long v, long long a) { return (v + a - 1) / a * a; }
static long long cdiv(long long a, long long b) { return (a + b - 1) / b; }

// CTA pairs of a B200.  The layout counts with this constant, so that a
// workspace's size is the descriptor's alone; launches ask the device.
constexpr int kPairs = 74;

// What a workspace starts on, and what the fp32 hidden planes need: their
// stores are 32 bytes wide.
constexpr size_t kWsAlign = 16, kHidAlign = 32;

// Where everything lies in the workspace, a function of the descriptor alone.
struct Layout {
  bool few;                  // forward of a few positions: hnd_ffn_few.cuh, operands token-major
  bool token, packed;        // token-major operands; samples gathered into rows of all positions
  int planes;
  long long batches, Lx;     // of the position axis as the products see it
  long long pitch;           // of packed rows (token: of a position's channels)
  long long hpitch;          // of a position's hidden channels
  size_t x, dy, w, hid, part, fold, bytes;
  long long act_plane, w_plane, hid_plane;   // elements
  int splits;                // of the weight gradients
  int cols, folds;           // of y and dx: columns of a tile, splits
};

// Columns of the tiles of a product of `N` columns over `m_tiles` tiles of 256
// rows: 256, unless there are fewer, or fewer tiles than half the pairs.
// Narrower tiles bring the rows of A in more often, so they are only taken
// where pairs would be idle (3 x 777 positions, C 200, F 536: 10 tiles, the
// second product 13 us with 256 columns, 9.3 with 64).
static int tile_cols(long long N, long long m_tiles) {
  int cols = 256;
  while (cols > 64 && (N <= cols / 2 || m_tiles * cdiv(N, cols) < kPairs / 2)) cols /= 2;
  return cols;
}

// Splits of the K loop of y or dx, where there are so few tiles that most
// pairs would be idle, each of eight stages at least: the partial sums are
// those of 74 tiles at most (9 positions, C 24, F 5280, fp32 training: one
// tile of 1000 stages, training 310 us unsplit, 118 so).
static int data_splits(long long tiles, long long stages) {
  const long long most = kPairs / tiles, deep = stages / 8;
  long long s = most < deep ? most : deep;
  if (s < 2) return 1;
  return static_cast<int>(cdiv(stages, cdiv(stages, s)));
}

// The most stages that one accumulator of a bf16 product adds up.  The tensor
// core cuts what it adds to an accumulator, always towards zero (fp32: see
// Params::piece), and over T positions the loss grows with T: sums of equal
// signs were off by 1.0e-3 at 9362 additions, 4.2e-3 at 43690, more than the
// result's own rounding.  4096 additions, 4 a stage, lose 4.5e-4; the other
// products' depth, 65536 channels at most (dx: twice), comes to the same or
// twice that.  (2^20 positions, C 256, F 1024: 6 splits before, 16 so, training
// 7.55 -> 7.67 ms.)
constexpr long long kDeepest = 1024;

// Splits of the weight gradients' K loops.  In stages of a pair (0.27 us at
// full rate): rounds of tiles, each with 8 stages' worth for a tile's ends;
// split, the partial sums go through memory once each way and one more
// kernel runs.  C 256, F 1024, 32768 positions: 6 splits, 12 tiles otherwise
// on 74 pairs; C 2048, F 5632: none (3 would add 67 us of partial sums).
static int weight_splits(long long C, long long F, long long stages) {
  const long long tiles = 2 * cdiv(C, 256) * cdiv(F, 256) + cdiv(F, 256) * cdiv(C, 256);
  int best = 1;
  long long cost = 0;
  for (int s = 1; s <= 32 && (s == 1 || stages / s >= 4); ++s) {
    const long long c = cdiv(tiles * s, kPairs) * (cdiv(stages, s) + 8) + (s > 1 ? 15 + s * C * F * 24 / 1750000 : 0);
    if (s == 1 || c < cost) best = s, cost = c;
  }
  return best;
}

static Layout layout(const FfnArgs& a, bool backward) {
  Layout l{};
  const long long T = a.B * a.L;
  l.planes = a.bf16 ? 1 : 3;
  l.token = a.L == 1;
  l.few = !backward && T <= kFewMost;
  // A row of positions has to start on 16 bytes for TMA, and a sample's last
  // tile of 256 positions should not be mostly empty: gathering costs one
  // pass over the activations, an empty half tile half the products.
  l.packed = !l.token && (!a.bf16 || a.L % 8 || (a.B > 1 && 4 * up(a.L, 256) > 5 * a.L));
  const bool merged = l.token || l.packed;
  l.batches = merged ? 1 : a.B;
  l.Lx = merged ? T : a.L;
  l.pitch = l.token ? a.C : up(T, 8);
  l.hpitch = a.bf16 ? a.F : up(a.F, 16);      // fp32: whole 32-byte stores
  const bool copied = l.packed || !a.bf16;
  // offsets are from the workspace rounded up to kHidAlign bytes (Ffn::ws)
  size_t at = 0;
  auto take = [&](long long elements, size_t size) {
    const size_t here = at;
    at += (static_cast<size_t>(elements) * size + 255) / 256 * 256;
    return here;
  };
  if (l.few) {      // activations gathered token-major unless they lie so, weights as they are
    l.act_plane = T * a.C;
    l.hid_plane = T * a.F;
    if (!l.token || !a.bf16) l.x = take(l.planes * l.act_plane, 2);
    l.hid = take(l.planes * l.hid_plane, 2);
    l.bytes = at;
    return l;
  }
  l.act_plane = l.token ? T * a.C : a.C * l.pitch;
  l.w_plane = a.C * a.F;
  l.hid_plane = l.batches * l.Lx * l.hpitch;
  if (copied) l.x = take(l.planes * l.act_plane, 2);
  if (copied && backward) l.dy = take(l.planes * l.act_plane, 2);
  if (!a.bf16) l.w = take(9 * l.w_plane, 2);
  l.hid = take((backward ? 3 : 1) * l.planes * l.hid_plane, 2);
  l.cols = tile_cols(a.C, l.batches * cdiv(l.Lx, 256));
  l.folds = data_splits(l.batches * cdiv(l.Lx, 256) * cdiv(a.C, l.cols), cdiv(a.F, kBK));
  if (l.folds > 1) l.fold = take(l.folds * l.batches * a.C * l.Lx, 4);
  l.splits = 1;
  if (backward) {
    // every split gets a stage at least
    const long long stages = l.batches * cdiv(l.Lx, kBK);
    long long per = cdiv(stages, weight_splits(a.C, a.F, stages * (a.bf16 ? 1 : 6)));
    if (a.bf16 && per > kDeepest) per = kDeepest;
    l.splits = static_cast<int>(cdiv(stages, per));
    if (l.splits > 1) l.part = take(3 * l.splits * l.w_plane, 4);
  }
  l.bytes = at + (a.bf16 ? 0 : kHidAlign - kWsAlign);
  return l;
}

size_t ffn_workspace(const FfnArgs& a, bool backward) { return layout(a, backward).bytes; }

// ---------------------------------------------------------------- tensor maps
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeFn encoder() {
  static const EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// A bf16 matrix in memory: `rows` rows of `inner` adjacent elements, `count` of them `batch` elements apart.
struct Mat {
  const void* p;
  long long inner, rows, count, pitch, batch;
};

static bool encode(CUtensorMap* map, const Mat& m, int box_inner, int box_rows, CUtensorMapSwizzle swizzle) {
  const EncodeFn fn = encoder();
  if (!fn) return false;
  const cuuint64_t dim[3] = {static_cast<cuuint64_t>(m.inner), static_cast<cuuint64_t>(m.rows),
                             static_cast<cuuint64_t>(m.count)};
  const cuuint64_t stride[2] = {static_cast<cuuint64_t>(m.pitch) * 2, static_cast<cuuint64_t>(m.batch) * 2};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t step[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(m.p), dim, stride, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// -------------------------------------------------------------------- launch
struct Launch {
  Params p{};
  int maps = 0, jobs = 0;
  bool ok = true;

  int add(const Mat& m, int box_inner, int box_rows, CUtensorMapSwizzle swizzle) {
    if (maps == kMaxMaps || !encode(&p.map[maps], m, box_inner, box_rows, swizzle)) {
      ok = false;
      return 0;
    }
    return maps++;
  }
  // an operand whose tile axis (m or n) is contiguous / whose k axis is
  int mn(const Mat& m) { return add(m, 64, kBK, CU_TENSOR_MAP_SWIZZLE_128B); }
  int km(const Mat& m, int rows = 128) { return add(m, kBK, rows, CU_TENSOR_MAP_SWIZZLE_128B); }
  int store(const Mat& m) { return add(m, 128, 32, CU_TENSOR_MAP_SWIZZLE_NONE); }
  // hidden rows of `wide` channels
  int store_hidden(const Mat& m, int wide) {
    return add(m, wide, 128, wide == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
  }
  void job(const Job& j) { p.job[jobs++] = j; }
};

template <int EPI, bool F32>
static cudaError_t run(Launch& l, cudaStream_t st) {
  if (!l.ok) return cudaErrorInvalidValue;
  long long tiles = 0;
  for (int i = 0; i < l.jobs; ++i) {
    Job& j = l.p.job[i];
    const long long per = static_cast<long long>(j.batches) * j.mt * j.nt;
    tiles += per * j.splits;
    if (tiles >= 1LL << 31) return cudaErrorInvalidValue;
    j.per = make_div(static_cast<uint32_t>(per));
    j.group8 = make_div(static_cast<uint32_t>(8 * j.nt));
    j.mdiv = make_div(static_cast<uint32_t>(j.mt));
  }
  l.p.tiles = static_cast<int>(tiles);
  auto kern = k_ffn_gemm<EPI, F32>;
  constexpr int smem = Plan<EPI, F32>::kSmem;
  static_assert(smem <= static_cast<int>(kMaxSmem), "shared memory");
  const cudaError_t e = ensure_smem(kern, smem);
  if (e != cudaSuccess) return e;
  long long pairs = sm_count() / 2;
  if (pairs > tiles) pairs = tiles;
  return launch_pdl(true, kern, dim3(static_cast<unsigned>(2 * pairs)), dim3(Plan<EPI, F32>::kThreads), smem, st, l.p);
}

template <bool F32, int NT, bool DUAL>
static cudaError_t run_few(const FewParams& p, bool early, cudaStream_t st) {
  // the depth over the warps: four chunks of 32 each where there is as much
  int warps = p.K / 128;
  warps = warps < 2 ? 2 : warps > (DUAL ? 8 : 16) ? (DUAL ? 8 : 16) : warps;
  const size_t smem = sizeof(float) * warps * (DUAL ? 2 : 1) * NT * 128;
  return launch_pdl(early, k_ffn_few<F32, NT, DUAL>, dim3(static_cast<unsigned>((p.rows + 15) / 16)),
                    dim3(static_cast<unsigned>(warps * 32)), smem, st, p);
}

template <bool F32, bool DUAL>
static cudaError_t run_few(const FewParams& p, bool early, cudaStream_t st) {
  return p.T <= 8    ? run_few<F32, 1, DUAL>(p, early, st)
         : p.T <= 16 ? run_few<F32, 2, DUAL>(p, early, st)
                     : run_few<F32, 4, DUAL>(p, early, st);
}

template <bool F32>
static cudaError_t forward_few(const FfnArgs& a) {
  using TT = typename std::conditional<F32, float, bf16>::type;
  const Layout l = layout(a, false);
  const int T = static_cast<int>(a.B * a.L), C = static_cast<int>(a.C), F = static_cast<int>(a.F);
  bf16* hid = reinterpret_cast<bf16*>(static_cast<char*>(a.ws) + l.hid);
  const bf16* x = static_cast<const bf16*>(a.x);
  if (!l.token || F32) {
    bf16* to = reinterpret_cast<bf16*>(static_cast<char*>(a.ws) + l.x);
    k_ffn_gather<TT><<<static_cast<unsigned>(cdiv(static_cast<long long>(T) * C, 256)), 256, 0, a.stream>>>(
        static_cast<const TT*>(a.x), to, C, static_cast<int>(a.L), T, l.act_plane);
    x = to;
  }
  FewParams h{};
  h.w0 = a.wg, h.w1 = a.wu, h.x = x, h.x_plane = l.act_plane;
  h.T = T, h.rows = F, h.K = C, h.act = a.act;
  h.hid = hid, h.hid_plane = l.hid_plane;
  cudaError_t e = run_few<F32, true>(h, false, a.stream);
  if (e != cudaSuccess) return e;
  FewParams y{};
  y.w0 = a.wd, y.x = hid, y.x_plane = l.hid_plane;
  y.T = T, y.rows = C, y.K = F;
  y.y = a.y, y.L = static_cast<int>(a.L);
  return run_few<F32, false>(y, true, a.stream);
}

template <bool F32>
struct Ffn {
  using TT = typename std::conditional<F32, float, bf16>::type;
  // columns of a tile: hidden channels, and columns of the other products
  using PG = Plan<kEpiGrad, F32>;
  static constexpr int hn = Plan<kEpiHidden, F32>::kCols, gn = PG::kCols;
  const FfnArgs& a;
  const Layout l;
  const long long T;
  Mat x, dy, wg, wu, wd, hid[3];

  char* ws(size_t at) const {
    const uintptr_t base = reinterpret_cast<uintptr_t>(a.ws);
    return reinterpret_cast<char*>(F32 ? (base + kHidAlign - 1) / kHidAlign * kHidAlign : base) + at;
  }
  bf16* wsb(size_t at) const { return reinterpret_cast<bf16*>(ws(at)); }

  Ffn(const FfnArgs& args, bool backward) : a(args), l(layout(args, backward)), T(args.B * args.L) {
    const bool copied = l.packed || F32;
    x = activation(copied ? ws(l.x) : a.x);
    dy = activation(copied ? ws(l.dy) : a.dy);
    const void* w[3] = {a.wg, a.wu, a.wd};
    if (F32)
      for (int i = 0; i < 3; ++i) w[i] = wsb(l.w) + 3 * i * l.w_plane;
    wg = weight(w[0], a.F, a.C), wu = weight(w[1], a.F, a.C), wd = weight(w[2], a.C, a.F);
    for (int i = 0; i < 3; ++i)
      hid[i] = Mat{wsb(l.hid) + i * l.planes * l.hid_plane, a.F, l.Lx, l.batches * l.planes, l.hpitch, l.Lx * l.hpitch};
  }
  Mat activation(const void* p) const {
    if (l.token) return Mat{p, a.C, T, l.planes, a.C, l.act_plane};
    if (l.packed) return Mat{p, T, a.C, l.planes, l.pitch, l.act_plane};
    return Mat{p, a.L, a.C, a.B, a.L, a.C * a.L};
  }
  Mat weight(const void* p, long long rows, long long cols) const { return Mat{p, cols, rows, l.planes, cols, l.w_plane}; }

  // Everything of the call that is not read where it lies.
  cudaError_t pack(bool backward) const {
    Packs packs{};
    int n = 0;
    long long most = 0;
    auto add = [&](const void* src, bf16* dst, long long B, long long rows, long long L, long long pitch, long long plane) {
      packs.p[n++] = Pack{src, dst, rows, L, B * L, pitch, plane};
      if (pitch / 8 * rows > most) most = pitch / 8 * rows;
    };
    const void* acts[2] = {a.x, a.dy};
    const size_t to[2] = {l.x, l.dy};
    for (int i = 0; i < (backward ? 2 : 1); ++i) {
      if (l.packed)
        add(acts[i], wsb(to[i]), a.B, a.C, a.L, l.pitch, l.act_plane);
      else if (F32)
        add(acts[i], wsb(to[i]), 1, T, a.C, a.C, l.act_plane);
    }
    const void* w[3] = {a.wg, a.wu, a.wd};
    for (int i = 0; F32 && i < 3; ++i) {
      const long long rows = i < 2 ? a.F : a.C, cols = i < 2 ? a.C : a.F;
      add(w[i], wsb(l.w) + 3 * i * l.w_plane, 1, rows, cols, cols, l.w_plane);
    }
    if (!n) return cudaSuccess;
    const long long blocks = cdiv(most, 256);
    k_ffn_pack<TT><<<dim3(static_cast<unsigned>(blocks < 148 * 8 ? blocks : 148 * 8), static_cast<unsigned>(n)), 256, 0,
                     a.stream>>>(packs);
    return cudaGetLastError();
  }

  Launch start() const {
    Launch n;
    n.p.act = a.act;
    n.p.piece = 4;
    n.p.status = a.status;
    // plane distances in the third coordinate: a batched operand has its batches in between
    n.p.a_plane = n.p.b_plane = 1;
    return n;
  }
  // activations as the rows of a product (m = positions): the position axis
  // is contiguous, except token-major, where the channels are
  int positions(Launch& n, const Mat& m) const { return l.token ? n.km(m) : n.mn(m); }
  Seg data_seg(int ma, int mb, bool a_mn, bool b_mn, int ncols, int acc, int clear) const {
    return Seg{ma, mb, mb, a_mn, b_mn, l.batches > 1, 0, ncols, ncols, ncols / 2, 0, acc, clear};
  }
  // G and U of `cols` hidden channels side by side: the first CTA brings Wg, the second Wu
  Seg gates_seg(Launch& n, int cols, int step) const {
    Seg s = data_seg(positions(n, x), n.km(wg, cols), !l.token, false, 2 * cols, 0, 1);
    s.b1 = n.km(wu, cols);
    s.nstep = step;
    s.noff = 0;
    return s;
  }
  Job data_job(int nseg, long long N, int per_tile, long long depth) const {
    Job j{};
    j.nseg = nseg;
    j.batches = static_cast<int>(l.batches);
    j.mt = static_cast<int>(cdiv(l.Lx, 256));
    j.nt = static_cast<int>(cdiv(N, per_tile));
    j.cols = per_tile;
    j.splits = j.kbatches = 1;
    j.kblocks = j.kper = static_cast<int>(cdiv(depth, kBK));
    j.M = l.Lx;
    j.N = N;
    return j;
  }
  void hidden_out(Launch& n, int count) const {
    for (int i = 0; i < count; ++i) {
      n.p.hid[i] = static_cast<bf16*>(const_cast<void*>(hid[i].p));
      if (!F32) n.p.hmap[i] = n.store_hidden(hid[i], count == 1 ? Plan<kEpiHidden, F32>::kWide : PG::kWide);
    }
    n.p.hid_plane = l.hid_plane;
    n.p.hid_rs = l.hpitch;
  }
  // y or dx: back to the activations' own layout
  void activation_out(Launch& n, Job& j, void* p) const {
    j.ptr = p;
    if (l.folds > 1) {
      j.splits = l.folds;
      j.kper = static_cast<int>(cdiv(j.kblocks, l.folds));
      j.kind = kOutF32;
      j.ptr = ws(l.fold);
      j.rs = l.Lx;
      j.bs = a.C * l.Lx;
      return;
    }
    if (l.token) {
      j.kind = kOutTok;
      j.rs = a.C;
    } else if (l.packed) {
      j.kind = F32 ? kOutF32 : kOutBf16;
      j.rs = a.L;
      j.group = a.L;
      j.gs = a.C * a.L;
    } else {
      j.kind = kOutTma;
      j.map = n.store(activation(p));
    }
  }

  cudaError_t fold(void* out) const {
    if (l.folds == 1) return cudaSuccess;
    const long long n = l.batches * a.C * l.Lx, blocks = cdiv(n, 256);
    k_ffn_fold<TT><<<static_cast<unsigned>(blocks < 148 * 8 ? blocks : 148 * 8), 256, 0, a.stream>>>(
        reinterpret_cast<const float*>(ws(l.fold)), static_cast<TT*>(out), a.C, a.L, l.Lx, n, l.folds, l.token);
    return cudaGetLastError();
  }

  cudaError_t forward() const {
    cudaError_t e;
    if ((e = pack(false)) != cudaSuccess) return e;
    Launch h = start();
    h.p.seg[0] = gates_seg(h, hn, hn);
    hidden_out(h, 1);
    h.job(data_job(1, a.F, hn, a.C));
    if ((e = run<kEpiHidden, F32>(h, a.stream)) != cudaSuccess) return e;
    Launch y = start();
    const int on = l.cols;
    y.p.seg[0] = data_seg(y.km(hid[0]), y.km(wd, on / 2), false, false, on, 0, 1);
    Job j = data_job(1, a.C, on, a.F);
    activation_out(y, j, a.y);
    y.job(j);
    e = run<kEpiOut, F32>(y, a.stream);
    return e == cudaSuccess ? fold(a.y) : e;
  }

  cudaError_t backward() const {
    cudaError_t e;
    if ((e = pack(true)) != cudaSuccess) return e;
    // H, dG, dU
    Launch h = start();
    if (F32) {
      h.p.seg[0] = gates_seg(h, gn, gn);
      h.p.seg[1] = data_seg(positions(h, dy), h.mn(wd), !l.token, true, gn, 2 * gn, 1);
    } else {      // dH of 256 channels, then G and U of 128 and of the other 128
      h.p.seg[0] = data_seg(positions(h, dy), h.mn(wd), !l.token, true, gn, 256, 1);
      h.p.seg[1] = h.p.seg[2] = gates_seg(h, 128, gn);
      h.p.seg[2].nbase = 128;
    }
    hidden_out(h, 3);
    h.job(data_job(F32 ? 2 : 3, a.F, gn, a.C));
    if ((e = run<kEpiGrad, F32>(h, a.stream)) != cudaSuccess) return e;
    // dX
    Launch d = start();
    d.p.piece = 2;      // of both its segments
    const int on = l.cols;
    d.p.seg[0] = data_seg(d.km(hid[1]), d.mn(wg), false, true, on, 0, 1);
    d.p.seg[1] = data_seg(d.km(hid[2]), d.mn(wu), false, true, on, 0, 0);
    Job j = data_job(2, a.C, on, a.F);
    activation_out(d, j, a.dx);
    d.job(j);
    if ((e = run<kEpiOut, F32>(d, a.stream)) != cudaSuccess || (e = fold(a.dx)) != cudaSuccess) return e;
    // dWg[f][c] = dG X', dWu[f][c] = dU X', dWd[c][f] = dY H'
    Launch w = start();
    const bool batched = l.batches > 1;
    const int stages = static_cast<int>(cdiv(l.Lx, kBK));
    const int cg = tile_cols(a.F, kPairs), cd = tile_cols(a.C, kPairs);
    const int mx = l.token ? w.mn(x) : w.km(x), mdy = l.token ? w.mn(dy) : w.km(dy, cd / 2);
    const int mh = w.mn(hid[0]), mdg = w.mn(hid[1]), mdu = w.mn(hid[2]);
    auto seg = [&](int ma, int mb, int a_mn, int b_mn, int cols) {
      return Seg{ma, mb, mb, a_mn, b_mn, batched, batched, cols, cols, cols / 2, 0, 0, 1};
    };
    w.p.seg[0] = seg(mx, mdg, l.token, 1, cg);
    w.p.seg[1] = seg(mx, mdu, l.token, 1, cg);
    w.p.seg[2] = seg(mh, mdy, 1, l.token, cd);
    void* out[3] = {a.dwg, a.dwu, a.dwd};
    float* part = reinterpret_cast<float*>(ws(l.part));
    for (int i = 0; i < 3; ++i) {
      Job q{};
      q.seg0 = i;
      q.nseg = 1;
      q.M = i < 2 ? a.C : a.F;
      q.N = i < 2 ? a.F : a.C;
      q.mt = static_cast<int>(cdiv(q.M, 256));
      q.cols = i < 2 ? cg : cd;
      q.nt = static_cast<int>(cdiv(q.N, q.cols));
      q.batches = 1;
      q.kbatches = static_cast<int>(l.batches);
      q.kblocks = stages;
      q.splits = l.splits;
      q.kper = static_cast<int>(cdiv(l.batches * stages, l.splits));
      q.rs = q.M;
      q.bs = l.w_plane;
      if (l.splits > 1) {
        q.kind = kOutF32;
        q.ptr = part + static_cast<size_t>(i) * l.splits * l.w_plane;
      } else if (F32) {
        q.kind = kOutF32;
        q.ptr = out[i];
      } else {
        q.kind = kOutTma;
        q.map = w.store(Mat{out[i], q.M, q.N, 1, q.M, l.w_plane});
      }
      w.job(q);
    }
    if ((e = run<kEpiOut, F32>(w, a.stream)) != cudaSuccess) return e;
    if (l.splits > 1) {
      const long long blocks = cdiv(l.w_plane, 1024);
      k_ffn_sum<TT><<<dim3(static_cast<unsigned>(blocks < 148 * 8 ? blocks : 148 * 8), 3), 256, 0, a.stream>>>(
          part, Sums{{a.dwg, a.dwu, a.dwd}}, l.w_plane, l.splits);
    }
    return cudaGetLastError();
  }
};

cudaError_t launch_ffn_forward(const FfnArgs& a) {
  if (a.B * a.L <= kFewMost) return a.bf16 ? forward_few<false>(a) : forward_few<true>(a);
  return a.bf16 ? Ffn<false>(a, false).forward() : Ffn<true>(a, false).forward();
}

cudaError_t launch_ffn_backward(const FfnArgs& a) {
  return a.bf16 ? Ffn<false>(a, true).backward() : Ffn<true>(a, true).backward();
}

}  // namespace hnd
