// Paged decode attention over a f32 cache, the forms for other calls (one file a format: they compile in parallel).
#include "paged_launch.cuh"

namespace coli {
namespace paged {

cudaError_t launch_f32_ext(const Params& p, int dp, int nt, int grid, cudaStream_t st) {
  return launch_format<DT_F32, true>(p, dp, nt, grid, st);
}

}  // namespace paged
}  // namespace coli
