// Sliding-window instantiations of the forward kernel, dense [B,H,S,D] and
// packed [T,H,D]: causal, with sinks and shared key heads.
//
// Mathematics: query i sees the keys j <= i with i - j < window or j < sinks, so
// a 128-query tile visits two runs of 128-key tiles, those with sinks and those
// its window reaches; masks apply to the tiles at the ends of the runs alone, as
// bits of 32 columns (a compare for each column and limit: 67.9 us in place of 65.5).
// Query head h reads key head h / group through the tensor map.
//
// Bound by the chain of a step (product, softmax, product), as in the causal
// kernel: (1, 32 heads, 4096 tokens, D = 128, bf16), window 1024, 4 sinks: 65.5
// us, 920 TFLOP/s of the visible pairs and 1130 of the tiles visited (a tile at each
// end of the window counts whole, and so does the one with sinks); tensor pipe
// 53 % active. Taking the first 32 keys alone of the tile with sinks gained 2 %
// and is not done. 16 packed sequences of 123 to 1994 tokens, 16
// heads on 4, window 512: 115 us, 662 TFLOP/s of the visible pairs and 975 of the
// tiles visited (an item visits 9 tiles where that prefill's visits 17, so its
// start and end, and the tile with sinks, weigh twice as much).
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
