// Paged decode attention over a bf16 cache (one file a format: they compile in parallel).
#include "paged_launch.cuh"

namespace coli {
namespace paged {

cudaError_t launch_bf16(const Params& p, int dp, int nt, int grid, cudaStream_t st) {
  return launch_format<DT_BF16>(p, dp, nt, grid, st);
}

}  // namespace paged
}  // namespace coli
