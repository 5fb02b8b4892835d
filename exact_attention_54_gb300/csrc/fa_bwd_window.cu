// Sliding-window instantiations of the backward pass, dense [B,H,S,D] and
// packed [T,H,D]: causal, with sinks and shared key heads.
#include "fa_bwd.cuh"

namespace fa {

cudaError_t launch_bwd_window(int D, bool bf16, bool varlen, const CUtensorMap *maps, const void *o,
                              const void *dout, const float *lse, void *dq, const BwdParams &p, cudaStream_t stream) {
#define FA_BWD(DD, BB, VV) \
    if (D == DD && bf16 == BB && varlen == VV) \
        return bwd::launch_t<DD, BB, true, VV, true>(maps, o, dout, lse, dq, p, stream);
    FA_BWD(64, false, false) FA_BWD(64, false, true) FA_BWD(64, true, false) FA_BWD(64, true, true)
    FA_BWD(128, false, false) FA_BWD(128, false, true) FA_BWD(128, true, false) FA_BWD(128, true, true)
#undef FA_BWD
    return cudaErrorInvalidValue;
}

}  // namespace fa
