// Writing keys and values into the paged 4-bit cache, and reading them back.
//
// Per group of 32 columns: s = max|x| / 7 rounded to 16 bits, n = x / s rounded
// to nearest even within [-7, 7]. Both kernels are streams (write: 2 D bytes
// read and D / 2 + D / 16 written per row; read: the reverse), bound by HBM
// bandwidth, or by launch latency for a few tokens.
//
// Grid: a chunk of tokens of one sequence per CTA (sequence = blockIdx.x /
// chunks), so that a token's sequence needs no search in cu_seqlens. D / 8
// lanes share a row of one key head, 8 columns (16 bytes) each; a thread takes
// the key row and the value row of the same token and head.
#include "fa_kv_q4.cuh"
#include "fa_launch.h"

namespace fa {
namespace q4 {

constexpr int kThreads = 256;
constexpr int kPasses = 4;  // rows per lane group and CTA, when a sequence has that many

// Tokens of one CTA: kPasses rows for each of its lane groups.
static int tokens_per_cta(int D, int Hkv) {
    const int rows = kPasses * kThreads / (D / 8);
    return Hkv >= rows ? 1 : rows / Hkv;
}

// The CTA's sequence and first token, checked; false if it has no work.
struct Chunk {
    int first, count;  // packed row of the first token; tokens
    long long pos;     // its position in the sequence
    const int *table;
};

__device__ __forceinline__ bool chunk_of(const KvQ4Params &p, Chunk &c) {
    const int b = static_cast<int>(blockIdx.x) / p.chunks;
    const int i0 = static_cast<int>(blockIdx.x) % p.chunks * p.tokens;
    const int t0 = p.cu_seqlens[b], t1 = p.cu_seqlens[b + 1];
    const int start = p.starts == nullptr ? 0 : p.starts[b];
    if (t0 < 0 || t1 < t0 || t1 > p.total || t1 - t0 > p.max_seqlen || start < 0) {
        if (threadIdx.x == 0) atomicExch(p.err, kDeviceErrSeqLens);
        return false;
    }
    c.first = t0 + i0;
    c.count = min(p.tokens, t1 - t0 - i0);
    c.pos = static_cast<long long>(start) + i0;
    c.table = p.block_table + static_cast<size_t>(b) * p.max_blocks;
    return c.count > 0;
}

// Row of the cache (in rows of a key head) that holds token i of the chunk, or
// -1 if the table names no page for it.
__device__ __forceinline__ long long cache_row(const KvQ4Params &p, const Chunk &c, int i, int h) {
    const long long pos = c.pos + i;
    const long long blk = pos >> p.log2_bs;
    const int page = blk < p.max_blocks ? c.table[blk] : -1;
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_blocks)) {
        atomicExch(p.err, kDeviceErrBadIndex);
        return -1;
    }
    return ((static_cast<long long>(page) * p.Hkv + h) << p.log2_bs) + (pos & ((1 << p.log2_bs) - 1));
}

template <int D, bool BF16>
__device__ __forceinline__ void quantise_row(const uint4 &x, uint8_t *codes, uint16_t *scales, long long row,
                                             int sub) {
    // max|x| of the group on the bits (16-bit floats without their sign order
    // like integers, infinities and NaNs last)
    uint32_t mx = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                           __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
    mx = max(mx & 0xffffu, mx >> 16);
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const bool finite = mx < (BF16 ? 0x7f80u : 0x7c00u);
    const uint16_t s16 = finite ? to16<BF16>(from16<BF16>(static_cast<uint16_t>(mx)) / 7.f) : uint16_t(0x7fff);
    const float s = from16<BF16>(s16);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t word = 0;  // nibble e: column 8 sub + e
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float v = from16<BF16>(static_cast<uint16_t>(w[e / 2] >> (16 * (e % 2))));
        // The quotient of two values of at most 11 bits is a tie or at least
        // 2^-12 (relative) away from one, so rounding it to fp32 first does
        // not change the integer it rounds to.
        const float n = s > 0.f ? fminf(fmaxf(rintf(v / s), -7.f), 7.f) : 0.f;
        word |= static_cast<uint32_t>(static_cast<int>(n) + 8) << (4 * e);
    }
    // Lane (w, c) of a row has columns 32 w + 8 c + (0..7): the 16 bits of
    // group w in pieces 2 c and 2 c + 1. The lanes of groups w and w ^ 1
    // exchange halves: even w keeps piece 2 c, odd w piece 2 c + 1, and each
    // stores one whole word.
    const int grp = sub / 4, c = sub % 4;
    const uint32_t other = __shfl_xor_sync(0xffffffffu, word, 4);
    const uint32_t out = grp % 2 == 0 ? __byte_perm(word, other, 0x5410) : __byte_perm(other, word, 0x7632);
    if (row >= 0) {
        uint32_t *dst = reinterpret_cast<uint32_t *>(codes + row * (D / 2));
        dst[(2 * c + grp % 2) * (D / 64) + grp / 2] = out;
        if (c == 0) scales[row * (D / kGroup) + grp] = s16;
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) fa_kv_write_q4_kernel(const KvQ4Params p) {
    Chunk c;
    if (!chunk_of(p, c)) return;
    constexpr int kLanes = D / 8;
    const int sub = threadIdx.x % kLanes;
    const int rows = c.count * p.Hkv;
    // whole warps run every pass: the group maxima are exchanged within a warp
    for (int r0 = 0; r0 < rows; r0 += kThreads / kLanes) {
        const int r = r0 + static_cast<int>(threadIdx.x) / kLanes;
        const bool there = r < rows;
        uint4 kx = make_uint4(0u, 0u, 0u, 0u), vx = kx;
        long long row = -1;
        if (there) {
            const size_t at = (static_cast<size_t>(c.first) * p.Hkv + r) * D + sub * 8;
            kx = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.k) + at));
            vx = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.v) + at));
            row = cache_row(p, c, r / p.Hkv, r % p.Hkv);
        }
        quantise_row<D, BF16>(kx, static_cast<uint8_t *>(p.k_codes), static_cast<uint16_t *>(p.k_scales), row, sub);
        quantise_row<D, BF16>(vx, static_cast<uint8_t *>(p.v_codes), static_cast<uint16_t *>(p.v_scales), row, sub);
    }
}

template <int D, bool BF16>
__device__ __forceinline__ uint4 read_row(const uint8_t *codes, const uint16_t *scales, long long row, int sub) {
    const int grp = sub / 4, c = sub % 4;
    const uint32_t *src = reinterpret_cast<const uint32_t *>(codes + row * (D / 2));
    const uint32_t a = src[2 * c * (D / 64) + grp / 2], b = src[(2 * c + 1) * (D / 64) + grp / 2];
    const float s = from16<BF16>(scales[row * (D / kGroup) + grp]);
    const uint32_t word = grp % 2 == 0 ? __byte_perm(a, b, 0x5410) : __byte_perm(a, b, 0x7632);
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lo = static_cast<float>(static_cast<int>((word >> (8 * i)) & 15u) - 8);
        const float hi = static_cast<float>(static_cast<int>((word >> (8 * i + 4)) & 15u) - 8);
        out[i] = ptx::pack2<BF16>(lo * s, hi * s);  // the fp32 product is exact: one rounding
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) fa_kv_read_q4_kernel(const KvQ4Params p) {
    Chunk c;
    if (!chunk_of(p, c)) return;
    constexpr int kLanes = D / 8;
    const int sub = threadIdx.x % kLanes;
    const int rows = c.count * p.Hkv;
    for (int r = static_cast<int>(threadIdx.x) / kLanes; r < rows; r += kThreads / kLanes) {
        const long long row = cache_row(p, c, r / p.Hkv, r % p.Hkv);
        if (row < 0) continue;
        const uint4 kx = read_row<D, BF16>(static_cast<const uint8_t *>(p.k_codes),
                                           static_cast<const uint16_t *>(p.k_scales), row, sub);
        const uint4 vx = read_row<D, BF16>(static_cast<const uint8_t *>(p.v_codes),
                                           static_cast<const uint16_t *>(p.v_scales), row, sub);
        const size_t at = (static_cast<size_t>(c.first) * p.Hkv + r) * D + sub * 8;
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.k) + at) = kx;
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.v) + at) = vx;
    }
}

template <int D, bool BF16>
static cudaError_t launch_t(bool write, const KvQ4Params &p, unsigned grid, cudaStream_t st) {
    if (write) fa_kv_write_q4_kernel<D, BF16><<<grid, kThreads, 0, st>>>(p);
    else fa_kv_read_q4_kernel<D, BF16><<<grid, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace q4

long long kv_q4_grid(int D, int num_seqs, KvQ4Params &p) {
    p.tokens = q4::tokens_per_cta(D, p.Hkv);
    p.chunks = (p.max_seqlen - 1) / p.tokens + 1;
    return static_cast<long long>(num_seqs) * p.chunks;
}

cudaError_t launch_kv_q4(int D, bool bf16, bool write, const KvQ4Params &p, int grid, cudaStream_t st) {
    const unsigned g = static_cast<unsigned>(grid);
    if (D == 64) return bf16 ? q4::launch_t<64, true>(write, p, g, st) : q4::launch_t<64, false>(write, p, g, st);
    return bf16 ? q4::launch_t<128, true>(write, p, g, st) : q4::launch_t<128, false>(write, p, g, st);
}

}  // namespace fa
