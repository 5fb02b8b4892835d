// Sliding-window instantiations of the backward pass, dense [B,H,S,D] and
// packed [T,H,D]: causal, with sinks and shared key heads.
//
// Mathematics: dV = P^T dO, dS = P (dP - D_i), dK = scale dS^T Q and dQ = scale
// dS K over the visible pairs; dK and dV of a shared key head are sums over its
// query heads, taken in one CTA's accumulators. A key tile takes the queries from
// its own position to the reach of its window, to the end if it holds sinks.
//
// Bound by the chain of a step (two products, softmax, three products), as in
// the causal kernel. 16 packed sequences of 123 to 1994 tokens, 16 heads on 4,
// D = 128, bf16, window 512, 4 sinks: 385 us, of which the row pass (D_i, zeroed
// dQ accumulator) 54 at 5.7 TB/s, the main kernel 279 (tensor pipe 46 % active;
// without sinks about 43 less), the conversion of dQ and the joining of segments,
// in one launch, 44. D = 64, (1, 32 heads, 4096 tokens, window 1024, 4 sinks): 180
// us, 0.21 of the bf16 rate: one buffer for S^T and dP^T, so the products and the
// key-row work take turns (tensor pipe 26 % active).
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
