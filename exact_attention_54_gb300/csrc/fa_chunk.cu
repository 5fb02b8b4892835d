// Instantiations of the chunk attention kernels over a paged cache: D in {64, 128}, fp16 and bf16.
#include "fa_chunk.cuh"

namespace fa {

cudaError_t launch_fwd_paged(int D, bool bf16, const CUtensorMap *maps, const ChunkParams &p, int grid,
                             cudaStream_t st) {
    if (D == 64) return bf16 ? chunk::launch_t<64, true>(maps, p, grid, st) : chunk::launch_t<64, false>(maps, p, grid, st);
    return bf16 ? chunk::launch_t<128, true>(maps, p, grid, st) : chunk::launch_t<128, false>(maps, p, grid, st);
}

}  // namespace fa
