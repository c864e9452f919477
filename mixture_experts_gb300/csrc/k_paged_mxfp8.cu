// Paged decode attention over a mxfp8 cache (one file a format: they compile in parallel).
#include "paged_launch.cuh"

namespace coli {
namespace paged {

cudaError_t launch_mxfp8(const Params& p, int dp, int nt, int grid, cudaStream_t st) {
  return launch_format<DT_MXFP8, false>(p, dp, nt, grid, st);
}

}  // namespace paged
}  // namespace coli
