// hnd_block_api.cu -- the C ABI declared in include/hyena_nd_block.h: argument
// checks and launches of the operators around the convolution.
#include "hyena_nd_block.h"
#include "hnd_block.h"
#include "hnd_bounds.cuh"
#include "hnd_launch.h"

#include <cmath>
#include <cstdint>
#include <initializer_list>

namespace hnd {

cudaError_t register_buffers(const BoundsList& list, int* status, cudaStream_t st) {
#ifdef HYENA_ND_BOUNDS
  if (!status) {
    const cudaError_t e = static_status_word(&status);
    if (e != cudaSuccess) return e;
  }
#endif
  return bounds_register(list, status, st);
}

}  // namespace hnd

namespace {

constexpr long long kMaxC = 65536;
constexpr long long kMaxPositions = 1LL << 31;
constexpr long long kMaxElements = 1LL << 40;
constexpr size_t kControlBytes = 256;

struct Span {
  const void* p;
  size_t bytes;
};

bool misaligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}

// No output overlaps an input or another output.
bool disjoint(std::initializer_list<Span> in, std::initializer_list<Span> out) {
  for (const Span* o = out.begin(); o != out.end(); ++o) {
    for (const Span& i : in)
      if (overlap(*o, i)) return false;
    for (const Span* q = o + 1; q != out.end(); ++q)
      if (overlap(*o, *q)) return false;
  }
  return true;
}

hyena_nd_status check_shape(const hyena_nd_block_shape* s) {
  if (!s || s->B < 1 || s->C < 1 || s->L < 1) return HYENA_ND_ERR_INVALID_ARG;
  if (s->io_dtype != HYENA_ND_F32 && s->io_dtype != HYENA_ND_BF16) return HYENA_ND_ERR_INVALID_ARG;
  if (s->C > kMaxC || s->B >= kMaxPositions || s->L >= kMaxPositions || s->B * s->L >= kMaxPositions ||
      s->B * s->L * s->C >= kMaxElements || s->B * s->C >= kMaxPositions)
    return HYENA_ND_ERR_UNSUPPORTED;
  return HYENA_ND_OK;
}

size_t act_bytes(const hyena_nd_block_shape* s) {
  return static_cast<size_t>(s->B) * s->C * s->L * (s->io_dtype == HYENA_ND_BF16 ? 2 : 4);
}

hyena_nd_status check_norm(const hyena_nd_norm& n, hnd::NormStage* out) {
  if (n.kind != HYENA_ND_NORM_NONE && n.kind != HYENA_ND_NORM_RMS && n.kind != HYENA_ND_NORM_LAYER)
    return HYENA_ND_ERR_INVALID_ARG;
  if (n.kind == HYENA_ND_NORM_NONE) {
    if (n.w || n.b) return HYENA_ND_ERR_INVALID_ARG;
  } else if (!(n.eps > 0.f) || !std::isfinite(n.eps)) {
    return HYENA_ND_ERR_INVALID_ARG;
  }
  if (misaligned(n.w, 4) || misaligned(n.b, 4)) return HYENA_ND_ERR_MISALIGNED;
  out->kind = n.kind;
  out->eps = n.eps;
  out->w = n.w;
  out->b = n.b;
  return HYENA_ND_OK;
}

hyena_nd_status check_drop(double p, const int64_t* rng, hnd::DropStage* out) {
  if (!(p >= 0.0 && p <= 1.0)) return HYENA_ND_ERR_INVALID_ARG;
  out->border = static_cast<unsigned>(std::floor(p * 65536.0 + 0.5));
  out->factor = out->border < 65536u ? static_cast<float>(65536.0 / (65536.0 - out->border)) : 0.f;
  out->rng = rng;
  if (out->border && !rng) return HYENA_ND_ERR_INVALID_ARG;
  if (misaligned(rng, 8)) return HYENA_ND_ERR_MISALIGNED;
  return HYENA_ND_OK;
}

hyena_nd_status cuda_status(cudaError_t e) { return e == cudaSuccess ? HYENA_ND_OK : HYENA_ND_ERR_CUDA; }

// The checked build's table of the call's buffers.
hyena_nd_status bounds(std::initializer_list<Span> spans, int* status, cudaStream_t st) {
  hnd::BoundsList bl;
  for (const Span& s : spans) bl.add(s.p, s.bytes);
  return cuda_status(hnd::register_buffers(bl, status, st));
}

// Nothing thrown leaves a C entry.
template <class Fn>
hyena_nd_status guarded(Fn fn) {
  try {
    return fn();
  } catch (...) {
    return HYENA_ND_ERR_CUDA;
  }
}

hyena_nd_status check_join(const hyena_nd_block_shape* s, const hyena_nd_join* j, hnd::JoinArgs* a) {
  hyena_nd_status st = check_shape(s);
  if (st != HYENA_ND_OK) return st;
  if (!j) return HYENA_ND_ERR_INVALID_ARG;
  if ((st = check_norm(j->post, &a->post)) != HYENA_ND_OK) return st;
  if ((st = check_norm(j->pre, &a->pre)) != HYENA_ND_OK) return st;
  if ((st = check_drop(j->p, j->rng, &a->drop)) != HYENA_ND_OK) return st;
  if (misaligned(j->gate, 4) || misaligned(j->scale, 4)) return HYENA_ND_ERR_MISALIGNED;
  a->B = s->B, a->C = s->C, a->L = s->L;
  a->bf16 = s->io_dtype == HYENA_ND_BF16;
  a->gate = j->gate;
  a->scale = j->scale;
  return HYENA_ND_OK;
}

size_t join_ws(const hyena_nd_block_shape* s) { return hnd::join_workspace(s->B, s->C, s->L, s->io_dtype == HYENA_ND_BF16); }

hyena_nd_status join_backward(const hyena_nd_block_shape* s, hnd::JoinArgs& a, void* ws, size_t ws_bytes) {
  const size_t act = act_bytes(s), C4 = 4 * static_cast<size_t>(s->C), BC4 = C4 * static_cast<size_t>(s->B);
  const size_t need = join_ws(s);
  for (const void* p : {a.x, a.y, a.dh, a.dn, static_cast<const void*>(a.dx), static_cast<const void*>(a.dy),
                        static_cast<const void*>(ws)})
    if (misaligned(p, 16)) return HYENA_ND_ERR_MISALIGNED;
  for (const float* p : {a.dpost_w, a.dpost_b, a.dgate, a.dscale, a.dpre_w, a.dpre_b})
    if (misaligned(p, 4)) return HYENA_ND_ERR_MISALIGNED;
  if (ws_bytes < need) return HYENA_ND_ERR_WORKSPACE_TOO_SMALL;
  if (!disjoint({{a.x, act}, {a.y, act}, {a.dh, act}, {a.dn, act}, {a.post.w, C4}, {a.post.b, C4}, {a.gate, BC4},
                 {a.scale, C4}, {a.pre.w, C4}, {a.pre.b, C4}, {a.drop.rng, 16}},
                {{a.dx, act}, {a.dy, act}, {a.dpost_w, C4}, {a.dpost_b, C4}, {a.dgate, BC4}, {a.dscale, C4},
                 {a.dpre_w, C4}, {a.dpre_b, C4}, {ws, need}}))
    return HYENA_ND_ERR_INVALID_ARG;
  a.ws = ws;
  return bounds({{a.x, act}, {a.y, act}, {a.dh, act}, {a.dn, act}, {a.post.w, C4}, {a.post.b, C4}, {a.gate, BC4},
                 {a.scale, C4}, {a.pre.w, C4}, {a.pre.b, C4}, {a.drop.rng, 16}, {a.dx, act}, {a.dy, act},
                 {a.dgate, BC4}, {ws, need}},
                nullptr, a.stream);
}

}  // namespace

#ifdef HYENA_ND_BOUNDS
// Reads one byte through the check.
static __global__ void k_bounds_probe(const unsigned char* p, unsigned char* out) { *HND_G(out) = *HND_G(p); }
#endif

extern "C" {

#ifdef HYENA_ND_BOUNDS
// For the tests of the checked build, which alone has it: registers the first
// `registered` bytes of `buffer` and the byte `out` without a status word, and
// reads byte `at` of the buffer, which has to be the caller's memory.
HYENA_ND_API hyena_nd_status hyena_nd_debug_bounds_probe(const void* buffer, size_t registered, size_t at, void* out,
                                                         void* cuda_stream) {
  return guarded([&] {
    const cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    const hyena_nd_status st = bounds({{buffer, registered}, {out, 1}}, nullptr, stream);
    if (st != HYENA_ND_OK) return st;
    k_bounds_probe<<<1, 1, 0, stream>>>(static_cast<const unsigned char*>(buffer) + at, static_cast<unsigned char*>(out));
    return cuda_status(cudaGetLastError());
  });
}
#endif

hyena_nd_status hyena_nd_norm_forward(const hyena_nd_block_shape* s, const hyena_nd_norm* norm, const void* x, void* n,
                                      void* cuda_stream) {
  return guarded([&] {
    hnd::JoinArgs a;
    hyena_nd_join j{};
    if (!norm || norm->kind == HYENA_ND_NORM_NONE) return HYENA_ND_ERR_INVALID_ARG;
    j.pre = *norm;
    hyena_nd_status st = check_join(s, &j, &a);
    if (st != HYENA_ND_OK) return st;
    if (!x || !n) return HYENA_ND_ERR_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(n, 16)) return HYENA_ND_ERR_MISALIGNED;
    const size_t act = act_bytes(s), C4 = 4 * static_cast<size_t>(s->C);
    if (!disjoint({{x, act}, {norm->w, C4}, {norm->b, C4}}, {{n, act}})) return HYENA_ND_ERR_INVALID_ARG;
    a.x = x;
    a.n = n;
    a.stream = static_cast<cudaStream_t>(cuda_stream);
    if ((st = bounds({{x, act}, {n, act}, {norm->w, C4}, {norm->b, C4}}, nullptr, a.stream)) != HYENA_ND_OK) return st;
    return cuda_status(hnd::launch_join_forward(a));
  });
}

hyena_nd_status hyena_nd_join_forward(const hyena_nd_block_shape* s, const hyena_nd_join* j, const void* x,
                                      const void* y, void* h, void* n, void* cuda_stream) {
  return guarded([&] {
    hnd::JoinArgs a;
    hyena_nd_status st = check_join(s, j, &a);
    if (st != HYENA_ND_OK) return st;
    if (!x || !y || !h || (n != nullptr) != (a.pre.kind != 0)) return HYENA_ND_ERR_INVALID_ARG;
    for (const void* p : {x, y, static_cast<const void*>(h), static_cast<const void*>(n)})
      if (misaligned(p, 16)) return HYENA_ND_ERR_MISALIGNED;
    const size_t act = act_bytes(s), C4 = 4 * static_cast<size_t>(s->C), BC4 = C4 * static_cast<size_t>(s->B);
    if (!disjoint({{x, act}, {y, act}, {j->post.w, C4}, {j->post.b, C4}, {j->gate, BC4}, {j->scale, C4},
                   {j->pre.w, C4}, {j->pre.b, C4}, {a.drop.rng, 16}},
                  {{h, act}, {n, act}}))
      return HYENA_ND_ERR_INVALID_ARG;
    a.x = x, a.y = y, a.h = h, a.n = n;
    a.stream = static_cast<cudaStream_t>(cuda_stream);
    if ((st = bounds({{x, act}, {y, act}, {h, act}, {n, act}, {j->post.w, C4}, {j->post.b, C4}, {j->gate, BC4},
                      {j->scale, C4}, {j->pre.w, C4}, {j->pre.b, C4}, {a.drop.rng, 16}},
                     nullptr, a.stream)) != HYENA_ND_OK)
      return st;
    return cuda_status(hnd::launch_join_forward(a));
  });
}

hyena_nd_status hyena_nd_norm_backward(const hyena_nd_block_shape* s, const hyena_nd_norm* norm, const void* x,
                                       const void* dn, void* dx, float* dw, float* db, void* ws, size_t ws_bytes,
                                       void* cuda_stream) {
  return guarded([&] {
    hnd::JoinArgs a;
    hyena_nd_join j{};
    if (!norm || norm->kind == HYENA_ND_NORM_NONE) return HYENA_ND_ERR_INVALID_ARG;
    j.pre = *norm;
    hyena_nd_status st = check_join(s, &j, &a);
    if (st != HYENA_ND_OK) return st;
    if (!x || !dn || !dx || !ws) return HYENA_ND_ERR_INVALID_ARG;
    a.x = x, a.dn = dn, a.dx = dx, a.dpre_w = dw, a.dpre_b = db;
    a.stream = static_cast<cudaStream_t>(cuda_stream);
    if ((st = join_backward(s, a, ws, ws_bytes)) != HYENA_ND_OK) return st;
    return cuda_status(hnd::launch_join_backward(a));
  });
}

hyena_nd_status hyena_nd_join_backward(const hyena_nd_block_shape* s, const hyena_nd_join* j, const void* x,
                                       const void* y, const void* dh, const void* dn, void* dx, void* dy,
                                       const hyena_nd_join_grads* grads, void* ws, size_t ws_bytes,
                                       void* cuda_stream) {
  return guarded([&] {
    hnd::JoinArgs a;
    hyena_nd_status st = check_join(s, j, &a);
    if (st != HYENA_ND_OK) return st;
    if (!x || !y || !dx || !dy || !ws || (dn != nullptr) != (a.pre.kind != 0)) return HYENA_ND_ERR_INVALID_ARG;
    a.x = x, a.y = y, a.dh = dh, a.dn = dn, a.dx = dx, a.dy = dy;
    if (grads) {
      a.dpost_w = grads->post_w, a.dpost_b = grads->post_b;
      a.dgate = grads->gate, a.dscale = grads->scale;
      a.dpre_w = grads->pre_w, a.dpre_b = grads->pre_b;
    }
    if (!a.pre.kind && (a.dpre_w || a.dpre_b)) return HYENA_ND_ERR_INVALID_ARG;
    if (!a.post.kind && (a.dpost_w || a.dpost_b)) return HYENA_ND_ERR_INVALID_ARG;
    a.stream = static_cast<cudaStream_t>(cuda_stream);
    if ((st = join_backward(s, a, ws, ws_bytes)) != HYENA_ND_OK) return st;
    return cuda_status(hnd::launch_join_backward(a));
  });
}

size_t hyena_nd_join_workspace_bytes(const hyena_nd_block_shape* s) {
  return check_shape(s) == HYENA_ND_OK ? join_ws(s) : 0;
}

hyena_nd_status hyena_nd_dropout(const hyena_nd_block_shape* s, double p, const int64_t* rng, const void* x, void* y,
                                 void* cuda_stream) {
  return guarded([&] {
    hyena_nd_status st = check_shape(s);
    if (st != HYENA_ND_OK) return st;
    hnd::DropStage d;
    if ((st = check_drop(p, rng, &d)) != HYENA_ND_OK) return st;
    if (!x || !y) return HYENA_ND_ERR_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(y, 16)) return HYENA_ND_ERR_MISALIGNED;
    const size_t act = act_bytes(s);
    if (!disjoint({{x, act}, {rng, 16}}, {{y, act}})) return HYENA_ND_ERR_INVALID_ARG;
    const cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    if ((st = bounds({{x, act}, {y, act}, {rng, 16}}, nullptr, stream)) != HYENA_ND_OK) return st;
    return cuda_status(
        hnd::launch_dropout(s->B * s->C * s->L, s->io_dtype == HYENA_ND_BF16, d, x, y, stream));
  });
}

static hyena_nd_status check_ffn(const hyena_nd_ffn* f, hnd::FfnArgs* a) {
  if (!f) return HYENA_ND_ERR_INVALID_ARG;
  const hyena_nd_status st = check_shape(&f->s);
  if (st != HYENA_ND_OK) return st;
  if (f->F < 1 || (f->act != HYENA_ND_ACT_SILU && f->act != HYENA_ND_ACT_GELU)) return HYENA_ND_ERR_INVALID_ARG;
  if (f->F > kMaxC || f->F % 8 || f->s.C % 8 || f->s.B * f->s.L * f->F >= kMaxElements)
    return HYENA_ND_ERR_UNSUPPORTED;
  a->B = f->s.B, a->C = f->s.C, a->L = f->s.L, a->F = f->F;
  a->bf16 = f->s.io_dtype == HYENA_ND_BF16;
  a->act = f->act;
  return HYENA_ND_OK;
}

size_t hyena_nd_ffn_workspace_bytes(const hyena_nd_ffn* f, int backward) {
  hnd::FfnArgs a;
  return check_ffn(f, &a) == HYENA_ND_OK ? hnd::ffn_workspace(a, backward != 0) : 0;
}

hyena_nd_status hyena_nd_ffn_forward(const hyena_nd_ffn* f, const void* x, const void* wg, const void* wu,
                                     const void* wd, void* y, void* control, void* ws, size_t ws_bytes,
                                     void* cuda_stream) {
  return guarded([&] {
    hnd::FfnArgs a;
    hyena_nd_status st = check_ffn(f, &a);
    if (st != HYENA_ND_OK) return st;
    if (!x || !wg || !wu || !wd || !y || !control || !ws) return HYENA_ND_ERR_INVALID_ARG;
    for (const void* p : {x, wg, wu, wd, static_cast<const void*>(y), static_cast<const void*>(control),
                          static_cast<const void*>(ws)})
      if (misaligned(p, 16)) return HYENA_ND_ERR_MISALIGNED;
    const size_t need = hnd::ffn_workspace(a, false);
    if (ws_bytes < need) return HYENA_ND_ERR_WORKSPACE_TOO_SMALL;
    const size_t act = act_bytes(&f->s), w = static_cast<size_t>(a.C) * a.F * (a.bf16 ? 2 : 4);
    if (!disjoint({{x, act}, {wg, w}, {wu, w}, {wd, w}}, {{y, act}, {ws, need}, {control, kControlBytes}}))
      return HYENA_ND_ERR_INVALID_ARG;
    a.x = x, a.wg = wg, a.wu = wu, a.wd = wd, a.y = y, a.ws = ws;
    a.status = static_cast<int*>(control);
    a.stream = static_cast<cudaStream_t>(cuda_stream);
    if ((st = bounds({{x, act}, {wg, w}, {wu, w}, {wd, w}, {y, act}, {ws, need}}, a.status, a.stream)) != HYENA_ND_OK)
      return st;
    return cuda_status(hnd::launch_ffn_forward(a));
  });
}

hyena_nd_status hyena_nd_ffn_backward(const hyena_nd_ffn* f, const void* x, const void* wg, const void* wu,
                                      const void* wd, const void* dy, void* dx, void* dwg, void* dwu, void* dwd,
                                      void* control, void* ws, size_t ws_bytes, void* cuda_stream) {
  return guarded([&] {
    hnd::FfnArgs a;
    hyena_nd_status st = check_ffn(f, &a);
    if (st != HYENA_ND_OK) return st;
    const void* all[] = {x, wg, wu, wd, dy, dx, dwg, dwu, dwd, control, ws};
    for (const void* p : all)
      if (!p) return HYENA_ND_ERR_INVALID_ARG;
    for (const void* p : all)
      if (misaligned(p, 16)) return HYENA_ND_ERR_MISALIGNED;
    const size_t need = hnd::ffn_workspace(a, true);
    if (ws_bytes < need) return HYENA_ND_ERR_WORKSPACE_TOO_SMALL;
    const size_t act = act_bytes(&f->s), w = static_cast<size_t>(a.C) * a.F * (a.bf16 ? 2 : 4);
    if (!disjoint({{x, act}, {wg, w}, {wu, w}, {wd, w}, {dy, act}},
                  {{dx, act}, {dwg, w}, {dwu, w}, {dwd, w}, {ws, need}, {control, kControlBytes}}))
      return HYENA_ND_ERR_INVALID_ARG;
    a.x = x, a.wg = wg, a.wu = wu, a.wd = wd, a.dy = dy;
    a.dx = dx, a.dwg = dwg, a.dwu = dwu, a.dwd = dwd, a.ws = ws;
    a.status = static_cast<int*>(control);
    a.stream = static_cast<cudaStream_t>(cuda_stream);
    if ((st = bounds({{x, act}, {wg, w}, {wu, w}, {wd, w}, {dy, act}, {dx, act}, {dwg, w}, {dwu, w}, {dwd, w},
                      {ws, need}},
                     a.status, a.stream)) != HYENA_ND_OK)
      return st;
    return cuda_status(hnd::launch_ffn_backward(a));
  });
}

}  // extern "C"
