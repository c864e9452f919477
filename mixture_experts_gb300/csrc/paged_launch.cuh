// Launch of one instantiation of the paged attention kernel.
#pragma once

#include "paged.cuh"

namespace coli {
namespace paged {


template <int FMT, int DP, int NT>
cudaError_t launch_main(const Params& p, int grid, cudaStream_t st) {
  using C = Cfg<FMT, DP, NT>;
  static bool ready[128] = {};  // the shared-memory limit is raised once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 128 || !ready[dev]) {
    e = cudaFuncSetAttribute(k_paged<FMT, DP, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 128) ready[dev] = true;
  }
  k_paged<FMT, DP, NT><<<grid, C::kWarps * 32, C::kSmem, st>>>(p);
  return cudaGetLastError();
}

// Head sizes run on the next of 64, 128, 256 (a smaller head's missing elements
// are never read from memory). Groups of more than 8 query heads take two
// column tiles where the registers hold them.
template <int FMT>
cudaError_t launch_format(const Params& p, int dp, int nt, int grid, cudaStream_t st) {
  if (dp == 64) {
    if constexpr (FMT != DT_F32)
      if (nt == 2) return launch_main<FMT, 64, 2>(p, grid, st);
    return launch_main<FMT, 64, 1>(p, grid, st);
  }
  if (dp == 128) {
    if constexpr (FMT != DT_F32)
      if (nt == 2) return launch_main<FMT, 128, 2>(p, grid, st);
    return launch_main<FMT, 128, 1>(p, grid, st);
  }
  if constexpr (FMT != DT_F32)
    if (nt == 2) return launch_main<FMT, 256, 2>(p, grid, st);
  return launch_main<FMT, 256, 1>(p, grid, st);
}

cudaError_t launch_f32(const Params& p, int dp, int nt, int grid, cudaStream_t st);
cudaError_t launch_bf16(const Params& p, int dp, int nt, int grid, cudaStream_t st);
cudaError_t launch_mxfp8(const Params& p, int dp, int nt, int grid, cudaStream_t st);
cudaError_t launch_mxfp4(const Params& p, int dp, int nt, int grid, cudaStream_t st);

}  // namespace paged
}  // namespace coli
