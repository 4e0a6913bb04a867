// The kernels of attend_paged_tiles.cuh for 64 channels: a file for each number of them, compiled side by side.
#include "attend_paged_tiles.cuh"

namespace hc {

cudaError_t launch_attend_paged_tiles_64(const AttendPagedParams& p, cudaStream_t s) { return launch_tiles<64>(p, s); }

}  // namespace hc
