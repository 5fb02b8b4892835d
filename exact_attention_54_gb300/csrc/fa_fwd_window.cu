// Sliding-window instantiations of the forward kernel, dense [B,H,S,D] and
// packed [T,H,D]: causal, with sinks and shared key heads.
#include "fa_fwd_kernel.cuh"

namespace fa {

cudaError_t launch_fwd_window(int D, bool bf16, bool varlen, const CUtensorMap *maps, const FwdParams &p, int grid,
                              cudaStream_t stream) {
#define FA_WINDOW(DD, BB, VV) \
    if (D == DD && bf16 == BB && varlen == VV) return launch_fwd_t<DD, BB, true, VV, true>(maps, p, grid, stream);
    FA_WINDOW(64, false, false) FA_WINDOW(64, false, true) FA_WINDOW(64, true, false) FA_WINDOW(64, true, true)
    FA_WINDOW(128, false, false) FA_WINDOW(128, false, true) FA_WINDOW(128, true, false) FA_WINDOW(128, true, true)
#undef FA_WINDOW
    return cudaErrorInvalidValue;
}

}  // namespace fa
