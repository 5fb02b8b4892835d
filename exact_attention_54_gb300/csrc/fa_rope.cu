// Rotary positions: rows of queries and keys with pairs of their columns turned
// by position-dependent angles (fa_rope, its gradient with inverse angles), and
// the same on the way into a paged 16-bit cache (fa_rope_kv_write).
//
// Pair i of a row, (a, b), at position p becomes m (a cos t - b sin t,
// b cos t + a sin t), t = p inv_freq[i]; the gradient is the same with -t. Every
// row is read and written once: a stream, bound by HBM, by launch latency for a
// few tokens.
//
// Angles: all heads of a token share them, so a CTA forms the cosines and sines
// of its tokens once, in shared memory. An angle in turns is the fraction of
// p inv_freq / 2 pi; far positions lose it in 32 bits (2^20 inv_freq is off by
// 2^-5 rad), so inv_freq / 2 pi is held as a 64-bit fraction and its product
// with p wraps as turns do: one integer product, off by 2^-63 p turns at
// most (inv_freq / 4 times that where it is above 4). The fraction's upper 32 bits, rounded to 24, go into sincospi.
//
// Grid: a chunk of tokens (x) of one sequence (y, z) per CTA, as in the 4-bit
// cache's kernels. D / 16 lanes share a row, two 16-byte pieces each: the
// pieces that pair up (half layout), or neighbouring ones.
//
// Measured: queries and keys of 21,915 tokens (32 and 8 heads of 128 columns) and their
// gradients, four calls, 143 us, 6.3 TB/s read and written; the same tokens into a cache
// 83 us, 6.4 TB/s; one token of 64 sequences 6 us. CTAs of 64 threads with two rows a
// lane group in flight: 32, 96 and 128 threads 150, 147 and 145 us, one row 148, four 152
// (registers then leave too few CTAs to cover the angles), twice the tokens 151. Rows are
// loaded ahead of the angles.
#include <math_constants.h>

#include "fa_kv_q4.cuh"
#include "fa_launch.h"

namespace fa {
namespace rope {

constexpr int kThreads = 64;
constexpr int kInFlight = 2;   // rows of a lane group with their loads in flight
constexpr int kMaxTokens = 8;  // of a CTA

// Two pieces of 8 columns of a row.
struct Pieces {
    uint4 a, b;
};

__device__ __forceinline__ uint32_t &word(uint4 &x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; }

// Turns the 8 pairs of a lane. turn: their (cos, sin), mscale in both, two pairs
// after another, then the next of the `lanes` lanes (with all of a lane's together a
// row's lanes read the same banks: 152 us for the four calls above).
// INTER: pairs are neighbouring columns of a (4) and b (4); else column i of a
// pairs with column i of b.
template <bool BF16, bool INTER>
__device__ __forceinline__ void rotate(Pieces &x, const float4 *turn, int lanes) {
    if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 t = turn[i * lanes];
            auto turn1 = [](uint32_t &w, float c, float s) {
                const float a = ptx::unpack_lo<BF16>(w), b = ptx::unpack_hi<BF16>(w);
                w = ptx::pack2<BF16>(a * c - b * s, b * c + a * s);
            };
            turn1(i < 2 ? word(x.a, 2 * i) : word(x.b, 2 * i - 4), t.x, t.y);
            turn1(i < 2 ? word(x.a, 2 * i + 1) : word(x.b, 2 * i - 3), t.z, t.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t &wa = word(x.a, i), &wb = word(x.b, i);
            const float a0 = ptx::unpack_lo<BF16>(wa), a1 = ptx::unpack_hi<BF16>(wa);
            const float b0 = ptx::unpack_lo<BF16>(wb), b1 = ptx::unpack_hi<BF16>(wb);
            const float4 t = turn[i * lanes];
            wa = ptx::pack2<BF16>(a0 * t.x - b0 * t.y, a1 * t.z - b1 * t.w);
            wb = ptx::pack2<BF16>(b0 * t.x + a0 * t.y, b1 * t.z + a1 * t.w);
        }
    }
}

// f / 2 pi without its whole part, in units of 2^-64: f is m 2^e, so it is m C 2^(e - 2)
// for C = 2^66 / 2 pi. (Double precision, of which GB300 has little, took 2 us more.)
__device__ __forceinline__ unsigned long long fraction_of_turn(float f) {
    const unsigned long long C = 0xa2f9836e4e44152aull;
    const uint32_t u = __float_as_uint(f);
    const int exponent = (u >> 23) & 255, shift = 152 - max(exponent, 1);
    const unsigned long long m = (u & 0x7fffff) | (exponent > 0 ? 0x800000 : 0);
    const unsigned long long hi = __umul64hi(m, C), lo = m * C;
    unsigned long long r;
    if (shift >= 64) r = shift < 128 ? hi >> (shift - 64) : 0;
    else if (shift > 0) r = hi << (64 - shift) | lo >> shift;
    else r = shift > -64 ? lo << -shift : 0;
    return u >> 31 ? 0 - r : r;
}

// Cosines and sines (times mscale) of `tokens` tokens, pos(i) the position of
// token i. The whole CTA calls it; ends synchronised.
template <class Pos>
__device__ __forceinline__ void fill_turns(const RopeParams &p, float2 *turns, int tokens, Pos pos) {
    const int pairs = p.rot_dim / 2;
    for (int i = threadIdx.x; i < pairs; i += kThreads) {
        const float freq = p.inv_freq[i];
        const unsigned long long frac = fraction_of_turn(freq);
        const float m = isfinite(freq) ? p.mscale : CUDART_NAN_F;  // (the fraction of such a frequency is 0)
        const int slot = 2 * (i % 8 / 2 * (pairs / 8) + i / 8) + i % 2;  // (see rotate)
        for (int t = 0; t < tokens; ++t) {
            const long long at = static_cast<long long>(static_cast<unsigned long long>(pos(t)) * frac);
            float s, c;
            sincospif(static_cast<float>(static_cast<int>(at >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31
            turns[t * pairs + slot] = make_float2(c * m, (p.inverse ? -s : s) * m);
        }
    }
    __syncthreads();
}

// Columns of a lane's two pieces, and whether they are turned.
struct Lane {
    int a, b;
    bool turned;
    __device__ __forceinline__ Lane(int sub, int rot_dim, bool inter) {
        turned = sub < rot_dim / 16;
        a = turned && !inter ? sub * 8 : sub * 16;
        b = turned && !inter ? rot_dim / 2 + sub * 8 : sub * 16 + 8;
    }
};

// Rows [0, rows) of a CTA, lane group by lane group: source(r) is where row r is
// read; target(r, dst, token) where it is written (dst NULL: nowhere) and which of
// the CTA's tokens turns it (-1: none, copied). ready() is called once, behind
// the first loads; what target and the turning need may be made there.
template <bool BF16, bool INTER, class Source, class Ready, class Target>
__device__ __forceinline__ void stream_rows(const RopeParams &p, const float2 *turns, int rows, Source source,
                                            Ready ready, Target target) {
    const int lanes = p.D / 16, groups = kThreads / lanes;
    const int sub = threadIdx.x % lanes, pairs = p.rot_dim / 2;
    const Lane l(sub, p.rot_dim, INTER);
    bool first = true;
    for (int r0 = threadIdx.x / lanes; first || r0 < rows; r0 += groups * kInFlight) {
        Pieces x[kInFlight];
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            if (r0 + i * groups >= rows) continue;
            const uint16_t *src = source(r0 + i * groups);
            x[i].a = __ldcs(reinterpret_cast<const uint4 *>(src + l.a));
            x[i].b = __ldcs(reinterpret_cast<const uint4 *>(src + l.b));
        }
        if (first) ready();
        first = false;
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            if (r0 + i * groups >= rows) continue;
            uint16_t *dst;
            int token;
            target(r0 + i * groups, dst, token);
            if (dst == nullptr) continue;
            if (l.turned && token >= 0)
                rotate<BF16, INTER>(x[i], reinterpret_cast<const float4 *>(turns + token * pairs) + sub, pairs / 8);
            *reinterpret_cast<uint4 *>(dst + l.a) = x[i].a;
            *reinterpret_cast<uint4 *>(dst + l.b) = x[i].b;
        }
    }
}

template <bool BF16, bool INTER>
__global__ void __launch_bounds__(kThreads) fa_rope_kernel(const RopeParams p) {
    extern __shared__ __align__(16) float2 turns[];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const long long b = static_cast<long long>(blockIdx.z) * gridDim.y + blockIdx.y;
    if (b >= p.num_seqs) return;
    const int s0 = static_cast<int>(blockIdx.x) * p.tokens, n = min(p.tokens, p.total - s0);
    const uint16_t *src0 = static_cast<const uint16_t *>(p.q) + b * p.q_batch + s0 * p.q_stride;
    uint16_t *dst0 = static_cast<uint16_t *>(p.q_out) + b * p.o_batch + s0 * p.o_stride;
    stream_rows<BF16, INTER>(
        p, turns, n * p.H,
        [&](int r) {
            const int t = r / p.H;
            return src0 + t * p.q_stride + (r - t * p.H) * p.q_head;
        },
        [&] {
            fill_turns(p, turns, n, [&](int t) -> long long {
                return p.positions == nullptr ? s0 + t : p.positions[b * p.total + s0 + t];
            });
        },
        [&](int r, uint16_t *&dst, int &token) {
            token = r / p.H;
            dst = dst0 + token * p.o_stride + (r - token * p.H) * p.o_head;
        });
}

template <bool BF16, bool INTER>
__global__ void __launch_bounds__(kThreads) fa_rope_kv_write_kernel(const RopeParams p) {
    extern __shared__ __align__(16) float2 turns[];
    __shared__ long long rows[kMaxTokens];  // first key head's cache row of each token, or -1
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const long long b = static_cast<long long>(blockIdx.z) * gridDim.y + blockIdx.y;
    if (b >= p.num_seqs) return;
    const int i0 = static_cast<int>(blockIdx.x) * p.tokens;
    const int t0 = p.cu_seqlens[b], t1 = p.cu_seqlens[b + 1];
    const int start = p.starts == nullptr ? 0 : p.starts[b];
    if (t0 < 0 || t1 < t0 || t1 > p.total || t1 - t0 > p.max_seqlen || start < 0) {
        if (threadIdx.x == 0) atomicExch(p.err, kDeviceErrSeqLens);
        return;
    }
    const int first = t0 + i0, n = min(p.tokens, t1 - t0 - i0);
    if (n <= 0) return;
    const long long pos0 = static_cast<long long>(start) + i0;
    const int per = p.H + 2 * p.Hkv;
    stream_rows<BF16, INTER>(
        p, turns, n * per,
        [&](int r) {
            const int t = r / per, h = r - t * per;
            const long long at = first + t;
            if (h < p.H) return static_cast<const uint16_t *>(p.q) + at * p.q_stride + static_cast<long long>(h) * p.D;
            if (h < p.H + p.Hkv)
                return static_cast<const uint16_t *>(p.k) + at * p.k_stride + static_cast<long long>(h - p.H) * p.D;
            return static_cast<const uint16_t *>(p.v) + at * p.v_stride + static_cast<long long>(h - p.H - p.Hkv) * p.D;
        },
        [&] {
            if (threadIdx.x < n) {
                const long long pos = pos0 + threadIdx.x, blk = pos >> p.log2_bs;
                const int page = blk < p.max_blocks ? p.block_table[b * p.max_blocks + blk] : -1;
                const bool ok = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_blocks);
                if (!ok) atomicExch(p.err, kDeviceErrBadIndex);
                rows[threadIdx.x] =
                    ok ? ((static_cast<long long>(page) * p.Hkv) << p.log2_bs) + (pos & ((1 << p.log2_bs) - 1)) : -1;
            }
            fill_turns(p, turns, n, [&](int t) -> long long {
                return p.positions == nullptr ? pos0 + t : p.positions[first + t];
            });
        },
        [&](int r, uint16_t *&dst, int &token) {
            const int t = r / per, h = r - t * per;
            if (h < p.H) {
                token = t;
                dst = static_cast<uint16_t *>(p.q_out) + (static_cast<long long>(first + t) * p.H + h) * p.D;
                return;
            }
            const bool value = h >= p.H + p.Hkv;
            const int hk = h - p.H - (value ? p.Hkv : 0);
            token = value ? -1 : t;
            dst = rows[t] < 0 ? nullptr
                              : static_cast<uint16_t *>(value ? p.v_cache : p.k_cache) +
                                    (rows[t] + (static_cast<long long>(hk) << p.log2_bs)) * p.D;
        });
}

}  // namespace rope

// Tokens of a CTA: about kInFlight rows for each of its lane groups twice over,
// so that the angles of a token (64 sincos at D = 128) are spread over all
// threads; fewer where there would be less than a wave of CTAs.
static int rope_tokens(long long sequences, long long longest, int rows_per_token, int D, int sms) {
    const int groups = rope::kThreads / (D / 16);
    long long t = (2LL * rope::kInFlight * groups + rows_per_token - 1) / rows_per_token;
    while (t > 1 && sequences * ((longest + t - 1) / t) < 4LL * sms) t /= 2;
    return static_cast<int>(t < 1 ? 1 : t < rope::kMaxTokens ? t : rope::kMaxTokens);
}

cudaError_t launch_rope(bool write, bool bf16, RopeParams p, int sms, cudaStream_t st) {
    const int rows = write ? p.H + 2 * p.Hkv : p.H;
    const int longest = write ? p.max_seqlen : p.total;
    p.tokens = rope_tokens(p.num_seqs, longest, rows, p.D, sms);
    const unsigned seqs = static_cast<unsigned>(p.num_seqs), y = seqs < 65535u ? seqs : 65535u;
    const dim3 grid(static_cast<unsigned>((longest - 1) / p.tokens + 1), y, (seqs + y - 1) / y);
    const int smem = p.tokens * p.rot_dim / 2 * static_cast<int>(sizeof(float2));  // at most 32 KB
    using Kernel = void (*)(RopeParams);
    static const Kernel kernels[2][2][2] = {
        {{rope::fa_rope_kernel<false, false>, rope::fa_rope_kernel<false, true>},
         {rope::fa_rope_kernel<true, false>, rope::fa_rope_kernel<true, true>}},
        {{rope::fa_rope_kv_write_kernel<false, false>, rope::fa_rope_kv_write_kernel<false, true>},
         {rope::fa_rope_kv_write_kernel<true, false>, rope::fa_rope_kv_write_kernel<true, true>}}};
    return launch_early(kernels[write][bf16][p.interleaved != 0], grid, rope::kThreads, static_cast<size_t>(smem), st, true,
                        p);
}

}  // namespace fa
