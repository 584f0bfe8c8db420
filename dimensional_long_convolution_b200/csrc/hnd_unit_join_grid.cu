// Instantiations of the join's persistent kernels on grids, with rows of whole
// vectors and ragged ones.
#include "hnd_host_util.h"
#include "hnd_join_grid.cuh"

namespace hnd {

constexpr size_t kGridSmem = 184 * 1024;     // the most a plan asks for (fp32 forward, one lane, 2048 channels)

// Vectors of 16 bytes in a row, the last maybe in part.
static long long row_vectors(const JoinArgs& a) {
  const int v = a.bf16 ? 8 : 4;
  return (a.L + v - 1) / v;
}

template <class TT, int K, bool RAG>
static cudaError_t fwd(const JoinArgs& a, const JoinDev& j, int w, unsigned blocks) {
  auto kern = grid::k_join_grid_fwd<TT, K, RAG>;
  const size_t smem = grid::smem_bytes(2, K, w, 16 / sizeof(TT), RAG);
  const cudaError_t e = ensure_smem(kern, kGridSmem);
  if (e != cudaSuccess) return e;
  const long long per = RAG ? (row_vectors(a) + w - 1) / w : row_vectors(a);
  kern<<<blocks, grid::kT, smem, a.stream>>>(j, w, make_div(static_cast<uint32_t>(per)), static_cast<int>(per * a.B),
                                             static_cast<const TT*>(a.x), static_cast<const TT*>(a.y),
                                             static_cast<TT*>(a.h), static_cast<TT*>(a.n));
  return cudaGetLastError();
}

template <class TT, int K, bool RAG>
static cudaError_t bwd(const JoinArgs& a, const JoinDev& j, int w, int chunks, unsigned blocks, float4* part) {
  auto kern = grid::k_join_grid_bwd<TT, K, RAG>;
  const size_t smem = grid::smem_bytes(4, K, w, 16 / sizeof(TT), RAG);
  const cudaError_t e = ensure_smem(kern, kGridSmem);
  if (e != cudaSuccess) return e;
  kern<<<blocks, grid::kT, smem, a.stream>>>(j, w, static_cast<int>(row_vectors(a)), chunks,
                                             static_cast<const TT*>(a.x), static_cast<const TT*>(a.y),
                                             static_cast<const TT*>(a.dh), static_cast<const TT*>(a.dn),
                                             static_cast<TT*>(a.dx), static_cast<TT*>(a.dy), part);
  return cudaGetLastError();
}

template <class TT, bool RAG>
static cudaError_t fwd_k(const JoinArgs& a, const JoinDev& j, int w, int K, unsigned blocks) {
  return K == 1 ? fwd<TT, 1, RAG>(a, j, w, blocks) : fwd<TT, 16 / sizeof(TT) == 8 ? 4 : 8, RAG>(a, j, w, blocks);
}
template <class TT, bool RAG>
static cudaError_t bwd_k(const JoinArgs& a, const JoinDev& j, int w, int K, int chunks, unsigned blocks, float4* part) {
  return K == 1 ? bwd<TT, 1, RAG>(a, j, w, chunks, blocks, part) : bwd<TT, 4, RAG>(a, j, w, chunks, blocks, part);
}

cudaError_t launch_join_grid_fwd(const JoinArgs& a, const JoinDev& j, int w, int K, unsigned blocks) {
  const bool ragged = a.L % (a.bf16 ? 8 : 4) != 0;
  if (a.bf16)
    return ragged ? fwd_k<__nv_bfloat16, true>(a, j, w, K, blocks) : fwd_k<__nv_bfloat16, false>(a, j, w, K, blocks);
  return ragged ? fwd_k<float, true>(a, j, w, K, blocks) : fwd_k<float, false>(a, j, w, K, blocks);
}

cudaError_t launch_join_grid_bwd(const JoinArgs& a, const JoinDev& j, int w, int K, int chunks, unsigned blocks,
                                 float4* part) {
  const bool ragged = a.L % (a.bf16 ? 8 : 4) != 0;
  if (a.bf16)
    return ragged ? bwd_k<__nv_bfloat16, true>(a, j, w, K, chunks, blocks, part)
                  : bwd_k<__nv_bfloat16, false>(a, j, w, K, chunks, blocks, part);
  return ragged ? bwd_k<float, true>(a, j, w, K, chunks, blocks, part)
                : bwd_k<float, false>(a, j, w, K, chunks, blocks, part);
}

}  // namespace hnd
