// Writing keys and values into the paged 4-bit cache, and reading them back.
//
// Per group of 32 columns: s = max|x| / 7 rounded to 16 bits, n = x / s rounded
// to nearest even within [-7, 7]. Both kernels are streams (write: 2 D bytes
// read and D / 2 + D / 16 written per row; read: the reverse), bound by HBM
// bandwidth, or by launch latency for a few tokens.
//
// Measured: reading 206 M values (100,527 tokens in 16 sequences, 8 key heads,
// D = 128) 84 us, 6.3 TB/s; writing the 45 M values of 16 prompts and reading
// them back 41 us, 5.0 TB/s, where instructions take as long as the bytes; a
// step of 64 tokens, written and read back, 10 us. CTAs of 128 threads: 256 and
// 512 lost 1 and 6 % on the prompts; one row per lane group lost 15 %, four 4 %;
// a lane took 8 columns before, 20 % slower; divisions by Hkv in the kernels, 8 %.
//
// Grid: a chunk of tokens (x) of one sequence (y, z) per CTA, so that a token's
// sequence needs no search in cu_seqlens and no division; the chunk's cache rows
// are looked up once, into shared memory. D / 16 lanes share a row of one key
// head, 16 columns each; a thread takes the key row and the value row of kPasses
// (token, head) pairs with all loads in flight.
#include "fa_kv_q4.cuh"
#include "fa_launch.h"

namespace fa {
namespace q4 {

constexpr int kThreads = 128;
constexpr int kPasses = 2;  // (token, head) pairs per lane group and CTA, when a sequence has that many
constexpr int kMaxTokens = kPasses * kThreads / 4;  // of a CTA: D = 64, one key head

// Tokens of one CTA: kPasses rows for each of its lane groups.
static int tokens_per_cta(int D, int Hkv) {
    const int rows = kPasses * kThreads / (D / 16);
    return Hkv >= rows ? 1 : rows / Hkv;
}

// The CTA's sequence and first token, checked; false if it has no work.
struct Chunk {
    int first, count;  // packed row of the first token; tokens
    long long pos;     // its position in the sequence
    const int *table;
};

__device__ __forceinline__ bool chunk_of(const KvQ4Params &p, Chunk &c) {
    const int b = static_cast<int>(blockIdx.z * gridDim.y + blockIdx.y);
    if (b >= p.num_seqs) return false;
    const int i0 = static_cast<int>(blockIdx.x) * p.tokens;
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

// First key head's cache row of each token of the chunk, or -1 if the table
// names no page for it (reported once: by the call that writes or reads it).
// The whole CTA calls it.
__device__ __forceinline__ void look_up(const KvQ4Params &p, const Chunk &c, long long *rows) {
    for (int i = threadIdx.x; i < c.count; i += kThreads) {
        const long long pos = c.pos + i, blk = pos >> p.log2_bs;
        const int page = blk < p.max_blocks ? c.table[blk] : -1;
        const bool ok = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_blocks);
        if (!ok) atomicExch(p.err, kDeviceErrBadIndex);
        rows[i] = ok ? ((static_cast<long long>(page) * p.Hkv) << p.log2_bs) + (pos & ((1 << p.log2_bs) - 1)) : -1;
    }
    __syncthreads();
}

// This lane group's (token, head) pairs: the first, then every step-th. The
// divisions by Hkv are the host's: first / Hkv is a product with inv_hkv, just
// above 2^31 / Hkv (exact while first * Hkv < 2^31: a CTA of several tokens has
// at most 2 kThreads pairs, of one token t = 0 and inv_hkv = 0).
struct Walk {
    int t, h;
    const KvQ4Params &p;
    __device__ __forceinline__ Walk(const KvQ4Params &p_, int first) : p(p_) {
        t = static_cast<int>(static_cast<unsigned long long>(first) * p.inv_hkv >> 31);
        h = first - t * p.Hkv;
    }
    __device__ __forceinline__ void next() {
        t += p.step_t;
        h += p.step_h;
        if (h >= p.Hkv) {
            h -= p.Hkv;
            ++t;
        }
    }
};

// 1 / x for normal x and 1 / x, relative error under 2^-22.
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Sixteen columns of a row, as a lane of the write kernel holds them.
struct Half {
    uint4 x[2];
};

// Codes (n + 8 in nibble e of word j: column 8 j + e of x) for scale s.
template <bool BF16>
__device__ __forceinline__ void quantise16(const Half &x, float s, uint32_t (&word)[2]) {
    // Where s is a normal number (and 1 / s is one): x / s is a tie n + 1/2 or
    // at least 2^-12 away from one, for x and s of at most 11 bits, and at most
    // 7.04. x * (1 / s), the reciprocal good to 2^-22, is off by less than
    // 2^-18, so rounding it to multiples of 2^-14 restores the ties and moves
    // nothing else across one; adding 1.5 2^23 + 8 then rounds to the nearest
    // even integer, which stands, plus 8, in the sum's low bits. The sum of
    // 16^e times those words (mod 2^32) holds the nibbles, but for a constant.
    // Two columns at a time.
    if (s >= (BF16 ? 1e-30f : 6.103515625e-5f)) {
        constexpr float kSnap = 768.f;          // 1.5 2^23 2^-14
        constexpr float kInt = 12582920.f;      // 1.5 2^23 + 8: bits 0x4b400008
        const float r = rcp_approx(s);
        const uint64_t inv = ptx::pk2(r, r), snap = ptx::pk2(kSnap, kSnap), less = ptx::pk2(-kSnap, -kSnap),
                       whole = ptx::pk2(kInt, kInt);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t w[4] = {x.x[j].x, x.x[j].y, x.x[j].z, x.x[j].w};
            word[j] = 0u - 0x4b400000u * 0x11111111u;
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const uint64_t v = ptx::pk2(from16<BF16>(static_cast<uint16_t>(w[e / 2])),
                                            from16<BF16>(static_cast<uint16_t>(w[e / 2] >> 16)));
                float n0, n1;
                ptx::upk2(ptx::fadd2(ptx::fadd2(ptx::ffma2(v, inv, snap), less), whole), n0, n1);
                word[j] += __float_as_uint(n0) * (1u << (4 * e)) + __float_as_uint(n1) * (1u << (4 * e + 4));
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        word[j] = 0;
#pragma unroll 1
        for (int e = 0; e < 8; ++e) {
            const uint32_t pair = e < 2 ? x.x[j].x : e < 4 ? x.x[j].y : e < 6 ? x.x[j].z : x.x[j].w;
            const float v = from16<BF16>(static_cast<uint16_t>(pair >> (16 * (e % 2))));
            const float n = s > 0.f ? fminf(fmaxf(rintf(v / s), -7.f), 7.f) : 0.f;
            word[j] |= static_cast<uint32_t>(static_cast<int>(n) + 8) << (4 * e);
        }
    }
}

// Codes and scales of a row. Lane sub = 2 w + h has columns 32 w + 16 h +
// (0..15) in x.
template <int D, bool BF16>
__device__ __forceinline__ void quantise_row(const Half &x, uint8_t *codes, uint16_t *scales, long long row, int sub) {
    // max|x| of the group on the bits (16-bit floats without their sign order
    // like integers, infinities and NaNs last)
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        mx = __vmaxu2(mx, __vmaxu2(x.x[i].x & 0x7fff7fffu, x.x[i].y & 0x7fff7fffu));
        mx = __vmaxu2(mx, __vmaxu2(x.x[i].z & 0x7fff7fffu, x.x[i].w & 0x7fff7fffu));
    }
    mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx & 0xffffu, mx >> 16);
    const bool finite = mx < (BF16 ? 0x7f80u : 0x7c00u);
    // max / 7 is no tie of 16-bit numbers (7 m with m odd has too many bits to
    // be one itself) and at least 1/7 of half a step away from each, so the
    // fp32 product with 1/7 rounds like the quotient.
    const uint16_t s16 =
        finite ? to16<BF16>(from16<BF16>(static_cast<uint16_t>(mx)) * (1.f / 7.f)) : uint16_t(0x7fff);
    uint32_t word[2];  // pieces 4 h, 4 h + 1 and 4 h + 2, 4 h + 3: 16 bits of group w each
    quantise16<BF16>(x, from16<BF16>(s16), word);  // a NaN scale takes the slow way: all n = 0
    // The lanes of groups w and w ^ 1 exchange a word: even w stores the first
    // two pieces, odd w the others, whole words.
    const int w = sub / 2, h = sub % 2;
    const bool odd = w % 2 != 0;
    const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? word[0] : word[1], 2);
    const uint32_t lo = odd ? other : word[0], hi = odd ? word[1] : other;
    if (row >= 0) {
        uint32_t *dst = reinterpret_cast<uint32_t *>(codes + row * (D / 2)) + (4 * h + 2 * (w % 2)) * (D / 64) + w / 2;
        dst[0] = __byte_perm(lo, hi, 0x5410);
        dst[D / 64] = __byte_perm(lo, hi, 0x7632);
        if (h == 0) scales[row * (D / kGroup) + w] = s16;
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) fa_kv_write_q4_kernel(const KvQ4Params p) {
    __shared__ long long rows[kMaxTokens];
    Chunk c;
    if (!chunk_of(p, c)) return;
    constexpr int kLanes = D / 16, kStep = kThreads / kLanes;
    const int sub = threadIdx.x % kLanes;
    const int pairs = c.count * p.Hkv;
    // whole warps run every pass: the group maxima are exchanged within a warp
    for (int r0 = 0; r0 < pairs; r0 += kPasses * kStep) {
        const int r = r0 + static_cast<int>(threadIdx.x) / kLanes;
        Half kx[kPasses], vx[kPasses];
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const bool there = r + i * kStep < pairs;
            const size_t at = (static_cast<size_t>(c.first) * p.Hkv + r + i * kStep) * D + sub * 16;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                kx[i].x[j] = vx[i].x[j] = make_uint4(0u, 0u, 0u, 0u);
                if (there) {
                    kx[i].x[j] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.k) + at) + j);
                    vx[i].x[j] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.v) + at) + j);
                }
            }
        }
        if (r0 == 0) look_up(p, c, rows);  // behind the loads
        Walk w(p, r);
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            if (r0 + i * kStep >= pairs) break;  // the same for the whole CTA
            const long long first = r + i * kStep < pairs ? rows[w.t] : -1;
            const long long row = first < 0 ? -1 : first + (static_cast<long long>(w.h) << p.log2_bs);
            quantise_row<D, BF16>(kx[i], static_cast<uint8_t *>(p.k_codes), static_cast<uint16_t *>(p.k_scales), row,
                                  sub);
            quantise_row<D, BF16>(vx[i], static_cast<uint8_t *>(p.v_codes), static_cast<uint16_t *>(p.v_scales), row,
                                  sub);
            w.next();
        }
    }
}

// A lane's words of a row as loaded, and its group's scale. Lane sub = 2 w + h
// loads two of the four pieces that hold columns 32 w + 16 h + (0..15), for
// its own group and the one that shares the words with it (see quantise_row).
struct Packed {
    uint32_t a, b;
    uint16_t s;
};

template <int D>
__device__ __forceinline__ Packed load_half(const uint8_t *codes, const uint16_t *scales, long long row, int sub) {
    const int w = sub / 2, h = sub % 2;
    const uint32_t *src =
        reinterpret_cast<const uint32_t *>(codes + row * (D / 2)) + (4 * h + 2 * (w % 2)) * (D / 64) + w / 2;
    return {src[0], src[D / 64], scales[row * (D / kGroup) + w]};
}

// s * n of the eight, rounded once: n is exact in either 16-bit type (u + 1024
// or u + 128, as masked into the mantissa, less 1032 or 136), so a 16-bit
// product is the rounded one.
template <bool BF16>
__device__ __forceinline__ uint4 unpack8(uint32_t word, uint16_t s) {
    uint32_t v[4];  // columns i and 4 + i
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = ((word >> (4 * i)) & 0x000f000fu) | (BF16 ? 0x43004300u : 0x64006400u);
        if constexpr (BF16) {
            const __nv_bfloat162 n = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&u),
                                             __bfloat162bfloat162(__ushort_as_bfloat16(0x4308)));  // 136
            const __nv_bfloat162 y = __hmul2_rn(n, __bfloat162bfloat162(__ushort_as_bfloat16(s)));
            v[i] = *reinterpret_cast<const uint32_t *>(&y);
        } else {
            const __half2 n = __hsub2(*reinterpret_cast<const __half2 *>(&u),
                                      __half2half2(__ushort_as_half(0x6408)));  // 1032
            const __half2 y = __hmul2_rn(n, __half2half2(__ushort_as_half(s)));
            v[i] = *reinterpret_cast<const uint32_t *>(&y);
        }
    }
    return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                      __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
}

// Sixteen columns of every lane's row; the whole warp calls it. `dst` NULL:
// not stored.
template <bool BF16>
__device__ __forceinline__ void store_half(uint16_t *dst, const Packed &x, int sub, bool v8, uint64_t policy) {
    const bool odd = sub / 2 % 2 != 0;
    const uint32_t lo = __byte_perm(x.a, x.b, 0x5410), hi = __byte_perm(x.a, x.b, 0x7632);
    const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 2);
    if (dst == nullptr) return;
    const uint4 y0 = unpack8<BF16>(odd ? other : lo, x.s), y1 = unpack8<BF16>(odd ? hi : other, x.s);
    if (v8) {
        const uint32_t y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
        ptx::st_global_v8_hint(dst, y, policy);
    } else {
        __stcs(reinterpret_cast<uint4 *>(dst), y0);
        __stcs(reinterpret_cast<uint4 *>(dst) + 1, y1);
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) fa_kv_read_q4_kernel(const KvQ4Params p) {
    __shared__ long long rows[kMaxTokens];
    Chunk c;
    if (!chunk_of(p, c)) return;
    constexpr int kLanes = D / 16, kStep = kThreads / kLanes;
    const int sub = threadIdx.x % kLanes;
    const int pairs = c.count * p.Hkv;
    const bool v8 = ((reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v)) & 31) == 0;
    const uint64_t policy = ptx::l2_policy_evict_first();
    look_up(p, c, rows);
    // whole warps run every pass: lanes exchange words
    for (int r0 = 0; r0 < pairs; r0 += kPasses * kStep) {
        const int r = r0 + static_cast<int>(threadIdx.x) / kLanes;
        Walk w(p, r);
        Packed k[kPasses], v[kPasses];
        bool there[kPasses];
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const long long first = r + i * kStep < pairs ? rows[w.t] : -1;
            there[i] = first >= 0;
            k[i] = v[i] = Packed{0u, 0u, 0};
            if (there[i]) {
                const long long row = first + (static_cast<long long>(w.h) << p.log2_bs);
                k[i] = load_half<D>(static_cast<const uint8_t *>(p.k_codes), static_cast<const uint16_t *>(p.k_scales),
                                    row, sub);
                v[i] = load_half<D>(static_cast<const uint8_t *>(p.v_codes), static_cast<const uint16_t *>(p.v_scales),
                                    row, sub);
            }
            w.next();
        }
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            if (r0 + i * kStep >= pairs) break;  // the same for the whole CTA
            const size_t at = (static_cast<size_t>(c.first) * p.Hkv + r + i * kStep) * D + sub * 16;
            store_half<BF16>(there[i] ? static_cast<uint16_t *>(p.k) + at : nullptr, k[i], sub, v8, policy);
            store_half<BF16>(there[i] ? static_cast<uint16_t *>(p.v) + at : nullptr, v[i], sub, v8, policy);
        }
    }
}

template <int D, bool BF16>
static cudaError_t launch_t(bool write, const KvQ4Params &p, dim3 grid, cudaStream_t st) {
    if (write) fa_kv_write_q4_kernel<D, BF16><<<grid, kThreads, 0, st>>>(p);
    else fa_kv_read_q4_kernel<D, BF16><<<grid, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace q4

long long kv_q4_grid(int D, int num_seqs, KvQ4Params &p) {
    const int step = q4::kThreads / (D / 16);
    p.num_seqs = num_seqs;
    p.tokens = q4::tokens_per_cta(D, p.Hkv);
    p.chunks = (p.max_seqlen - 1) / p.tokens + 1;
    p.inv_hkv = p.tokens == 1 ? 0u : (1u << 31) / static_cast<unsigned>(p.Hkv) + 1u;
    p.step_t = step / p.Hkv;
    p.step_h = step % p.Hkv;
    return static_cast<long long>(num_seqs) * p.chunks;
}

cudaError_t launch_kv_q4(int D, bool bf16, bool write, const KvQ4Params &p, cudaStream_t st) {
    // sequences over y and z (at most 65535 each)
    const unsigned seqs = static_cast<unsigned>(p.num_seqs), y = seqs < 65535u ? seqs : 65535u;
    const dim3 g(static_cast<unsigned>(p.chunks), y, (seqs + y - 1) / y);
    if (D == 64) return bf16 ? q4::launch_t<64, true>(write, p, g, st) : q4::launch_t<64, false>(write, p, g, st);
    return bf16 ? q4::launch_t<128, true>(write, p, g, st) : q4::launch_t<128, false>(write, p, g, st);
}

}  // namespace fa
