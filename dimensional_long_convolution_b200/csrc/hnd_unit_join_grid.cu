// Instantiations of the join on aligned grids.
#include "hnd_host_util.h"
#include "hnd_join_grid.cuh"

namespace hnd {

template <class TT, int K>
static cudaError_t fwd(const JoinArgs& a, const JoinDev& j, int w, unsigned blocks) {
  auto kern = grid::k_join_grid_fwd<TT, K>;
  const size_t smem = grid::smem_bytes(2, K, a.C, w, 16 / sizeof(TT));
  const cudaError_t e = ensure_smem(kern, grid::smem_bytes(2, K, 2048, 32, 16 / sizeof(TT)));
  if (e != cudaSuccess) return e;
  const long long per = a.L * sizeof(TT) / 16;
  kern<<<blocks, grid::kT, smem, a.stream>>>(j, w, make_div(static_cast<uint32_t>(per)), static_cast<int>(per * a.B),
                                             static_cast<const TT*>(a.x), static_cast<const TT*>(a.y), static_cast<TT*>(a.h), static_cast<TT*>(a.n));
  return cudaGetLastError();
}

template <class TT, int K>
static cudaError_t bwd(const JoinArgs& a, const JoinDev& j, int w, int chunks, unsigned blocks, float4* part) {
  auto kern = grid::k_join_grid_bwd<TT, K>;
  const size_t smem = grid::smem_bytes(4, K, a.C, w, 16 / sizeof(TT));
  const cudaError_t e = ensure_smem(kern, grid::smem_bytes(4, K, 2048, 32, 16 / sizeof(TT)));
  if (e != cudaSuccess) return e;
  kern<<<blocks, grid::kT, smem, a.stream>>>(j, w, static_cast<int>(a.L * sizeof(TT) / 16), chunks, static_cast<const TT*>(a.x), static_cast<const TT*>(a.y),
                                             static_cast<const TT*>(a.dh), static_cast<const TT*>(a.dn),
                                             static_cast<TT*>(a.dx), static_cast<TT*>(a.dy), part);
  return cudaGetLastError();
}

cudaError_t launch_join_grid_fwd(const JoinArgs& a, const JoinDev& j, int w, int K, unsigned blocks) {
  if (a.bf16) return K == 1 ? fwd<__nv_bfloat16, 1>(a, j, w, blocks) : fwd<__nv_bfloat16, 4>(a, j, w, blocks);
  return K == 1 ? fwd<float, 1>(a, j, w, blocks) : fwd<float, 8>(a, j, w, blocks);
}

cudaError_t launch_join_grid_bwd(const JoinArgs& a, const JoinDev& j, int w, int K, int chunks, unsigned blocks,
                                 float4* part) {
  if (a.bf16)
    return K == 1 ? bwd<__nv_bfloat16, 1>(a, j, w, chunks, blocks, part)
                  : bwd<__nv_bfloat16, 4>(a, j, w, chunks, blocks, part);
  return K == 1 ? bwd<float, 1>(a, j, w, chunks, blocks, part) : bwd<float, 4>(a, j, w, chunks, blocks, part);
}

}  // namespace hnd
