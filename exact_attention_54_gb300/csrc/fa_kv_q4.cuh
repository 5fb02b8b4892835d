// The row format of the paged 4-bit cache (include/fa.h): groups of 32
// columns with a 16-bit scale s, codes n + 8 in nibbles, value s * n.
//
// A row of D / 2 code bytes consists of eight pieces of D / 16 bytes. Piece g
// holds, for each group w, the four columns 32 w + 4 g + (0..3) in 16 bits. A
// thread that owns the same four columns of every group (the value side of
// the decode kernel) so reads one contiguous piece, and four lanes that share
// a row (its key side) read two pieces each; halves of a word always belong to
// different groups, so one byte permutation pairs two keys or two pieces.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sm103_ptx.cuh"

namespace fa {
namespace q4 {

constexpr int kGroup = 32;  // columns per scale

template <bool BF16>
__device__ __forceinline__ float from16(uint16_t x) {
    if constexpr (BF16) return __uint_as_float(static_cast<uint32_t>(x) << 16);
    else return __half2float(__ushort_as_half(x));
}

template <bool BF16>
__device__ __forceinline__ uint16_t to16(float x) {
    if constexpr (BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
    else return __half_as_ushort(__float2half_rn(x));
}

}  // namespace q4
}  // namespace fa
