// Shared by the paged decode kernels whose query heads come in groups that
// share a key head (fa_decode_gqa.cu: 16-bit pages, fa_decode_q4.cu: the 4-bit
// cache): the visible keys of a sequence, the tensor-core instructions, and the
// merge of warps and partitions.
//
// Split-KV as in fa_decode.cu: a unit is a sequence, a key head and up to 8 NT
// of its query heads; a CTA takes parts of units (see Plan), its warps stream
// tiles of keys and keep partial (m, l, O) each; the last part of a unit to
// finish merges its query heads.
//
// Fragments of mma.m16n8k16, lane = 4 g + c: the S^T = K Q^T product's A rows
// are 16 keys, of which a lane holds two (g and g + 8); its columns may come in
// any order that Q shares, so a lane reads contiguous bytes of its keys' rows.
// S^T's result (keys g, g + 8; heads 2c, 2c + 1) becomes the B operand (keys
// 2c, 2c + 1, 2c + 8, 2c + 9; head g) of O^T += V^T P^T by a transpose of 8x8
// 16-bit values (movmatrix); V^T's rows are columns of V that a lane picks so
// as to read contiguous bytes, and byte permutations pair the values of
// neighbouring keys.
//
// Why mma.sync and not tcgen05.mma: a group has few query heads. 8 columns fit
// a group as they are, where tcgen05.mma would pad it to the 64 or 128 rows of
// its smallest tile and take keys through shared memory in another layout.
#pragma once

#include <math_constants.h>

#include "fa_kv_q4.cuh"
#include "fa_launch.h"

namespace fa {
namespace gqa {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr float kMoveMax = 8.f;  // m moves when a score exceeds it by this (base-2 units)
constexpr float kNoMax = -3.402823466e38f;  // m before any key: below every score, and -inf - m stays -inf
constexpr unsigned kFull = 0xffffffffu;

// ------------------------------------------------------------ instructions --

// D = A B + C, fp32 sums.
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    mma16816<BF16>(d, a0, a1, a2, a3, b0, b1, d[0], d[1], d[2], d[3]);
}

// The transpose of an 8x8 matrix of 16-bit values: lane 4 g + c gives row g,
// columns 2c and 2c + 1, and receives column g, rows 2c and 2c + 1.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// N consecutive 32-bit words from global memory, read once.
template <int N>
__device__ __forceinline__ void load_words(uint32_t *r, const void *p) {
    if constexpr (N == 4)
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "l"(p));
    else if constexpr (N == 2)
        asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "l"(p));
    else
        asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(r[0]) : "l"(p));
}

// Two fp16 values: a - b.
__device__ __forceinline__ uint32_t sub16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// N consecutive 32-bit words from shared memory.
template <int N>
__device__ __forceinline__ void shared_words(uint32_t *r, uint32_t at) {
    if constexpr (N == 4)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(at)
                     : "memory");
    else if constexpr (N == 2)
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(at) : "memory");
    else
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r[0]) : "r"(at) : "memory");
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) { return ptx::pack2<BF16>(lo, hi); }

// ---------------------------------------------------------------- key list --

// The tiles of TILE keys (aligned) of a sequence that hold visible keys, in a
// list: first those that hold sinks, then those the window reaches.
template <int TILE>
struct KeyList {
    int L, w_lo, n_sink;  // length; the window starts here; sinks in front of it
    int sink_tiles, w_tile;
    int n;                // tiles in the list

    __device__ __forceinline__ KeyList(const GqaDecodeParams &p, int b) {
        L = min(max(p.seq_lens[b], 0), p.max_blocks << p.log2_bs);
        w_lo = p.window > 0 ? max(L - p.window, 0) : 0;
        n_sink = min(p.sinks, w_lo);
        sink_tiles = (n_sink + TILE - 1) / TILE;
        w_tile = max(w_lo / TILE, sink_tiles);
        n = sink_tiles + max((L + TILE - 1) / TILE - w_tile, 0);
    }
    __device__ __forceinline__ int key0(int i) const { return (i < sink_tiles ? i : i - sink_tiles + w_tile) * TILE; }
    __device__ __forceinline__ bool sees(int key) const { return key < L && (key >= w_lo || key < n_sink); }
    // any of the 16 keys from `key` on
    __device__ __forceinline__ bool sees16(int key) const { return key < L && (key + 16 > w_lo || key < n_sink); }
};

// ------------------------------------------------------------------- plan --

// A part of a unit: list entries [lo, hi) of its keys' tiles; the slot-th of
// `parts` parts.
struct Part {
    size_t bh0;  // first query head, in [B * H]
    int b, hk, heads, unit;
    int lo, hi, slot, parts;
    int live;    // 0: there is no part left
};

constexpr int kPlanSeqs = 512;  // sequences the balanced plan holds

// How the units' tiles are dealt out. Balanced: all units' tiles in a row are
// cut into equal runs, one per CTA of a single wave, so that sequences of any
// lengths keep every SM busy to the end; every CTA works the cut out for
// itself from seq_lens. A run is long enough that no unit falls into more than
// num_splits parts. Plain (one partition, more sequences than the plan holds,
// or little work): CTA x is partition x % num_splits of unit x / num_splits.
// It lives in shared memory: the kernels need their registers.
template <int TILE, int HT>
struct Plan {
    // what a unit's start costs, in tiles (4 bits, 8 key heads: 16 sequences of
    // 16384 to 32768 keys 120.7 -> 118.2 us, 64 of 1000 to 8000 101.7 -> 94.2 us;
    // 8 and 16 are worse by up to 2 %)
    static constexpr unsigned kStart = 12;
    unsigned prefix[kPlanSeqs + 1];  // balanced: tiles of one key head of the sequences before b
    unsigned run, at, end;           // balanced: tiles per CTA; this CTA's (all units' tiles fit 32 bits)
    Part part;

    __device__ __forceinline__ static int units_per_seq(const GqaDecodeParams &p) {
        return p.Hkv * ((p.group + HT - 1) / HT);
    }

    // The CTA's run; the whole CTA calls it.
    __device__ __forceinline__ void make(const GqaDecodeParams &p) {
        if (!p.balanced) {
            if (threadIdx.x == 0) {
                at = blockIdx.x;
                end = at + 1;
            }
            __syncthreads();
            return;
        }
        // a unit starts with kStart tiles that are not there: a CTA whose run
        // straddles units has that much less to read, and a sequence without
        // keys still gets a part, which writes its result
        for (int b = threadIdx.x; b < p.B; b += kThreads) prefix[b + 1] = KeyList<TILE>(p, b).n + kStart;
        __syncthreads();
        if (threadIdx.x < 32) {
            const int each = (p.B + 31) / 32, b0 = threadIdx.x * each;
            unsigned sum = 0, most = 0;
            for (int b = b0; b < min(b0 + each, p.B); ++b) {
                sum += prefix[b + 1];
                most = max(most, prefix[b + 1]);
            }
            unsigned before = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const unsigned v = __shfl_up_sync(kFull, before, off);
                if (static_cast<int>(threadIdx.x) >= off) before += v;
            }
            const unsigned total = __shfl_sync(kFull, before, 31) * units_per_seq(p);
            before -= sum;
            for (int b = b0; b < min(b0 + each, p.B); ++b) prefix[b + 1] = before += prefix[b + 1];
            most = __reduce_max_sync(kFull, most);
            if (threadIdx.x == 0) {
                prefix[0] = 0;
                run = (total + gridDim.x - 1) / gridDim.x;
                run = max(run, (most + p.num_splits - 2) / (p.num_splits - 1));
                run = max(run, 128u / TILE);  // a few keys for every warp
                at = static_cast<unsigned>(min(static_cast<unsigned long long>(blockIdx.x) * run,
                                               static_cast<unsigned long long>(total)));
                end = total - at > run ? at + run : total;
            }
        }
        __syncthreads();
    }

    // Puts this CTA's next part into `part`; the whole CTA calls it.
    __device__ __forceinline__ void next(const GqaDecodeParams &p) {
        if (threadIdx.x == 0) {
            const unsigned units_b = units_per_seq(p);
            part.live = at < end;
            if (at < end) {
                unsigned in_seq;  // unit within its sequence
                if (p.balanced) {
                    int b = 0;
                    for (int step = kPlanSeqs / 2; step > 0; step >>= 1)
                        if (b + step < p.B && prefix[b + step] * units_b <= at) b += step;
                    const unsigned n = prefix[b + 1] - prefix[b], first = prefix[b] * units_b;
                    in_seq = (at - first) / n;
                    const unsigned start = first + in_seq * n;
                    part.b = b;
                    const int lo = at - start, hi = min(end - start, n);
                    part.lo = max(lo - static_cast<int>(kStart), 0);
                    part.hi = max(hi - static_cast<int>(kStart), 0);
                    part.slot = blockIdx.x - start / run;
                    part.parts = (start + n - 1) / run - start / run + 1;
                    at = start + hi;
                } else {
                    const int unit = static_cast<int>(blockIdx.x) / p.num_splits;
                    part.b = unit / units_b;
                    in_seq = unit % units_b;
                    part.slot = static_cast<int>(blockIdx.x) % p.num_splits;
                    part.parts = p.num_splits;
                    const int n = KeyList<TILE>(p, part.b).n, per = (n + p.num_splits - 1) / p.num_splits;
                    part.lo = static_cast<int>(min(static_cast<long long>(part.slot) * per, static_cast<long long>(n)));
                    part.hi = min(part.lo + per, n);
                    at = end;
                }
                const int tiles_h = (p.group + HT - 1) / HT, h0 = in_seq % tiles_h * HT;
                part.hk = in_seq / tiles_h;
                part.heads = min(HT, p.group - h0);
                part.unit = part.b * units_b + in_seq;
                part.bh0 = static_cast<size_t>(part.b) * p.H + static_cast<size_t>(part.hk) * p.group + h0;
            }
        }
        __syncthreads();
    }
};

// ------------------------------------------------------------------- merge --

// The end of a part: the warps' shares (sm_m, sm_l, sm_o; written, not yet
// synchronised) become the part's, or the result where the unit is one part;
// then the last part to finish merges them all. Ends synchronised.
template <int D, bool BF16, int HT>
__device__ __forceinline__ void merge(const GqaDecodeParams &p, const Part &job, const float (*sm_m)[HT],
                                      const float (*sm_l)[HT], const float (*sm_o)[HT][D]) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int splits = job.parts, s = job.slot, heads = job.heads, unit = job.unit;
    const int stride = p.num_splits;
    const size_t bh0 = job.bh0;
    __syncthreads();
    // Result of one head, from parts (m, l, O) with weights 2^(m - M): no
    // visible key gives O = 0 and LSE = -inf, a NaN stays one.
    auto finish = [&](size_t bh, int d, float M, float Lw, float4 O) {
        const float inv = Lw == 0.f ? 0.f : 1.f / Lw;
        const uint2 out = make_uint2(pack16<BF16>(O.x * inv, O.y * inv), pack16<BF16>(O.z * inv, O.w * inv));
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.o) + bh * D + d) = out;
        if (d == 0) p.lse[bh] = Lw == 0.f ? -CUDART_INF_F : (M + log2f(Lw)) * 0.69314718055994531f;
    };
    for (int i = threadIdx.x; i < heads * (D / 4); i += kThreads) {
        const int h = i / (D / 4), d = i % (D / 4) * 4;
        float M = -CUDART_INF_F, Lw = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w][h]);
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = M == -CUDART_INF_F ? 1.f : ptx::ex2(sm_m[w][h] - M);
            const float4 v = *reinterpret_cast<const float4 *>(&sm_o[w][h][d]);
            Lw = fmaf(f, sm_l[w][h], Lw);
            O.x = fmaf(f, v.x, O.x);
            O.y = fmaf(f, v.y, O.y);
            O.z = fmaf(f, v.z, O.z);
            O.w = fmaf(f, v.w, O.w);
        }
        if (splits == 1) {
            finish(bh0 + h, d, M, Lw, O);
        } else {
            const size_t at = (bh0 + h) * stride + s;
            *reinterpret_cast<float4 *>(p.o_part + at * D + d) = O;
            if (d == 0) {
                p.m_part[at] = M;
                p.l_part[at] = Lw;
            }
        }
    }
    // ---- the last part of these heads merges them: a warp per head ----
    __shared__ int is_last;
    __syncthreads();
    if (splits == 1) return;
    if (threadIdx.x == 0) {
        // the barriers order the CTA's writes before this thread's fence, and
        // its second fence before the CTA's reads
        __threadfence();
        is_last = atomicAdd(p.counters + unit, 1) == splits - 1;
        __threadfence();
    }
    __syncthreads();
    if (!is_last) return;
    for (int h = warp; h < heads; h += kWarps) {
        const size_t at = (bh0 + h) * stride;
        float M = -CUDART_INF_F;
        for (int j = lane; j < splits; j += 32) M = fmaxf(M, __ldcg(p.m_part + at + j));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, off));
        float Lw = 0.f;
        constexpr int kLanes = D / 4, kRows = 32 / kLanes;  // lanes per row of 4-column pieces; rows per step
        const int d = lane % kLanes * 4, sub = lane / kLanes;
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j0 = 0; j0 < splits; j0 += 32) {
            const int j = j0 + lane;
            const float f = j >= splits ? 0.f : M == -CUDART_INF_F ? 1.f : ptx::ex2(__ldcg(p.m_part + at + j) - M);
            if (j < splits) Lw = fmaf(f, __ldcg(p.l_part + at + j), Lw);
            const int n = min(32, splits - j0);
#pragma unroll 4
            for (int k = 0; k < n; k += kRows) {
                const float fk = __shfl_sync(kFull, f, (k + sub) & 31);
                if (k + sub < n) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.o_part + (at + j0 + k + sub) * D + d));
                    O.x = fmaf(fk, v.x, O.x);
                    O.y = fmaf(fk, v.y, O.y);
                    O.z = fmaf(fk, v.z, O.z);
                    O.w = fmaf(fk, v.w, O.w);
                }
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) Lw += __shfl_xor_sync(kFull, Lw, off);
        if constexpr (kRows == 2) {
            O.x += __shfl_xor_sync(kFull, O.x, 16);
            O.y += __shfl_xor_sync(kFull, O.y, 16);
            O.z += __shfl_xor_sync(kFull, O.z, 16);
            O.w += __shfl_xor_sync(kFull, O.w, 16);
        }
        if (sub == 0) finish(bh0 + h, d, M, Lw, O);
    }
    if (threadIdx.x == 0) p.counters[unit] = 0;
}

}  // namespace gqa
}  // namespace fa
