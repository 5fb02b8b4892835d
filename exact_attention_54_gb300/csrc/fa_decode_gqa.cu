// One-token attention over a paged cache whose key heads are shared by groups
// of query heads, with a sliding window and sinks: 16-bit pages
// (fa_decode_paged_window) or the 4-bit cache (fa_decode_paged_q4).
//
// Split-KV as in fa_decode.cu: partial (m, l, O) per partition of the visible
// keys, the last partition of a key head to finish merges its query heads.
//
// Mathematics. With the scores x_j = scale q . k_j in base-2 units, a warp
// keeps per query head a running maximum m, l = sum_j 2^(x_j - m) and O =
// sum_j 2^(x_j - m) v_j over its keys; m is moved only when a score exceeds it
// by 2^8. The 4-bit cache holds k = s (u - 8), u a nibble, and s per 32
// columns w, so x = sum_w s_w (sum_d q_d u_d - 8 sum_d q_d): the second sum
// does not depend on the key, and a nibble is a number as it stands. Masked
// out of its word, nibble 0 of a 16-bit lane is the fp16 number u 2^-24, and
// nibble 1 is 16 u 2^-24 (below the normal numbers, which the tensor core takes
// exactly), so unpacking two values costs one logical operation; the factor
// 16 goes into q. V likewise: O = sum_j (p_j s_j) u_j - 8 sum_j (p_j s_j), both
// sums from the tensor core with the same rounded weights p_j s_j.
//
// Why this form: the keys and values of a group of query heads are read once
// (HBM bound), so each value read meets up to 8 query heads: 2 * 8 FMA per
// value and SM at HBM speed is beyond the FMA pipes, and 4-bit values would
// cost an instruction each to convert. mma.sync with keys as the 16 rows and
// 8 query heads as columns takes the fragments straight from the registers
// that the loads fill: nothing passes through shared memory, and no tile has
// to be padded to the 128 rows of tcgen05.mma.
//
// Fragments of mma.m16n8k16, lane = 4 g + c: the S^T product's A rows are keys
// g and g + 8 of a 16-key tile; its columns may come in any order that Q
// shares, so a lane loads contiguous bytes of its key's row. S^T's result
// (keys g, g + 8; heads 2c, 2c + 1) becomes the second product's B operand
// (keys 2c, 2c + 1, 2c + 8, 2c + 9; head g) by one 8x8 transpose of 16-bit
// pairs (movmatrix); its A operand pairs the values of neighbouring keys by
// byte permutations.
#include <math_constants.h>

#include "fa_kv_q4.cuh"
#include "fa_launch.h"

namespace fa {
namespace gqa {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr float kMoveMax = 8.f;       // m moves when a score exceeds it by this (base-2 units)
constexpr float kMostWeight = 4096.f; // 4-bit: largest rounded weight before its factor r is chosen again
constexpr float kMostFactor = 1.2676506002282294e30f;  // 2^100: r before any weight is known
constexpr unsigned kFull = 0xffffffffu;

// ------------------------------------------------------------ instructions --

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8x8 matrix of 16-bit values: lane 4 g + c gives row g,
// columns 2c and 2c + 1, and receives column g, rows 2c and 2c + 1.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
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

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) { return ptx::pack2<BF16>(lo, hi); }

// ------------------------------------------------------------------- tiles --

// The 16-key tiles of a sequence that hold visible keys, in a list: first
// those that hold sinks, then those the window reaches.
struct KeyList {
    int L, w_lo, n_sink;  // length; the window starts here; sinks in front of it
    int sink_tiles, w_tile;
    int n;                // tiles in the list

    __device__ __forceinline__ KeyList(const GqaDecodeParams &p, int b) {
        L = min(max(p.seq_lens[b], 0), p.max_blocks << p.log2_bs);
        w_lo = p.window > 0 ? max(L - p.window, 0) : 0;
        n_sink = min(p.sinks, w_lo);
        sink_tiles = (n_sink + 15) >> 4;
        w_tile = max(w_lo >> 4, sink_tiles);
        n = sink_tiles + max(((L + 15) >> 4) - w_tile, 0);
    }
    __device__ __forceinline__ int key0(int i) const { return (i < sink_tiles ? i : i - sink_tiles + w_tile) << 4; }
    __device__ __forceinline__ bool sees(int key) const { return key < L && (key >= w_lo || key < n_sink); }
};

template <int D, bool Q4, int NT = 1>
struct Shape {
    static constexpr int kW = D / 32;                     // column groups
    static constexpr int kKWords = Q4 ? D / 32 : D / 8;   // words of a key row per lane
    static constexpr int kVWords = Q4 ? D / 64 : D / 16;  // words of a value row per lane
    static constexpr int kSWords = D / 64;                // words of a row's scales
    static constexpr int kRowBytes = Q4 ? D / 2 : 2 * D;
    static constexpr int kMTiles = D / 16;                // 16-column tiles of O^T
    // tiles in flight per warp: a 4-bit tile is 2.3 KB (D = 128), a 16-bit one 8 KB
    static constexpr int kDepth = Q4 && NT == 1 ? 2 : 1;
    static constexpr int kCtas = NT == 1 ? 3 : 2;  // per SM
};

// A tile as its loads left it: keys g and g + 8 (k, and the scale rows of
// keys and values), values of keys 2c, 2c + 1, 2c + 8, 2c + 9 (v).
template <int D, bool Q4>
struct Tile {
    using S = Shape<D, Q4>;
    uint32_t k[2][S::kKWords];
    uint32_t v[4][S::kVWords];
    uint32_t ks[Q4 ? 2 : 1][S::kSWords], vs[Q4 ? 2 : 1][S::kSWords];
    int key0;
    bool whole;        // every key of the tile is visible (the same for the warp)
    uint32_t kin, vin; // else: bit i, whether this lane's i-th key row (value row) is
};

// Where this lane finds a tile: its page's first row of the tile (pages of 16
// keys and more), or the row of each of its keys.
template <int D, bool Q4>
struct Reader {
    using S = Shape<D, Q4>;
    const GqaDecodeParams &p;
    const KeyList &list;
    const int *table;
    int hk, g, c;
    bool bad_page;

    __device__ __forceinline__ long long row_of(int key, bool &ok) {
        ok = list.sees(key);
        if (!ok) return 0;
        const int page = table[key >> p.log2_bs];
        ok = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_blocks);
        if (!ok) {
            bad_page = true;
            return 0;
        }
        return ((static_cast<long long>(page) * p.Hkv + hk) << p.log2_bs) + (key & ((1 << p.log2_bs) - 1));
    }

    // The tile at key0, whose page is `page` (pages of 16 keys and more). Rows
    // that are not to be read are replaced by row 0 of the cache and masked.
    __device__ __forceinline__ void load(Tile<D, Q4> &t, int key0, int page) {
        t.key0 = key0;
        const char *kb = static_cast<const char *>(p.k), *vb = static_cast<const char *>(p.v);
        const char *ksb = static_cast<const char *>(p.ks), *vsb = static_cast<const char *>(p.vs);
        long long kr[2], vr[4];
        if (p.log2_bs >= 4) {
            const bool ok = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_blocks);
            bad_page |= !ok;
            const long long row = ok ? ((static_cast<long long>(page) * p.Hkv + hk) << p.log2_bs) +
                                           (key0 & ((1 << p.log2_bs) - 1))
                                     : 0;
            t.whole = ok && key0 >= list.w_lo && key0 + 16 <= list.L;
            if (!t.whole) {
                t.kin = t.vin = 0;
#pragma unroll
                for (int i = 0; i < 2; ++i) t.kin |= (ok && list.sees(key0 + g + 8 * i) ? 1u : 0u) << i;
#pragma unroll
                for (int i = 0; i < 4; ++i) t.vin |= (ok && list.sees(key0 + 2 * c + (i & 1) + 4 * (i & 2)) ? 1u : 0u) << i;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) kr[i] = row + g + 8 * i;
#pragma unroll
            for (int i = 0; i < 4; ++i) vr[i] = row + 2 * c + (i & 1) + 4 * (i & 2);
        } else {
            t.whole = false;
            t.kin = t.vin = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                bool ok;
                kr[i] = row_of(key0 + g + 8 * i, ok);
                t.kin |= (ok ? 1u : 0u) << i;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                bool ok;
                vr[i] = row_of(key0 + 2 * c + (i & 1) + 4 * (i & 2), ok);
                t.vin |= (ok ? 1u : 0u) << i;
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const char *row = kb + kr[i] * S::kRowBytes;
            if constexpr (Q4) {
                load_words<S::kKWords>(t.k[i], row + c * (D / 8));
                load_words<S::kSWords>(t.ks[i], ksb + kr[i] * (D / 16));
                load_words<S::kSWords>(t.vs[i], vsb + kr[i] * (D / 16));
            } else {
#pragma unroll
                for (int u = 0; u < S::kKWords / 4; ++u) load_words<4>(&t.k[i][4 * u], row + (c + 4 * u) * 16);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const char *row = vb + vr[i] * S::kRowBytes;
            if constexpr (Q4) {
                load_words<S::kVWords>(t.v[i], row + g * (D / 16));
            } else {
#pragma unroll
                for (int u = 0; u < S::kVWords / 4; ++u) load_words<4>(&t.v[i][4 * u], row + (g + 8 * u) * 16);
            }
        }
    }
};

// ------------------------------------------------------------------ kernel --

// grid: ((b * Hkv + key head) * head tiles + head tile) * num_splits +
// partition; a head tile is 8 NT query heads of the group.
template <int D, bool BF16, bool Q4, int NT>
__global__ void __launch_bounds__(kThreads, (Shape<D, Q4, NT>::kCtas)) fa_decode_gqa_kernel(const GqaDecodeParams p) {
    using S = Shape<D, Q4, NT>;
    constexpr int W = S::kW, MT = S::kMTiles, HT = 8 * NT;
    constexpr bool kMmaBf16 = BF16 && !Q4;  // 4-bit operands are fp16 numbers whatever the cache's type
    const int splits = p.num_splits;
    const int s = static_cast<int>(blockIdx.x) % splits, unit = static_cast<int>(blockIdx.x) / splits;
    const int tiles_h = (p.group + HT - 1) / HT;
    const int h0 = unit % tiles_h * HT, bk = unit / tiles_h;  // first query head of the group; sequence and key head
    const int b = bk / p.Hkv, hk = bk % p.Hkv;
    const int heads = min(HT, p.group - h0);
    const size_t bh0 = static_cast<size_t>(b) * p.H + static_cast<size_t>(hk) * p.group + h0;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int g = lane / 4, c = lane % 4;

    const KeyList list(p, b);
    const int per = (list.n + splits - 1) / splits;
    const int lo = static_cast<int>(min(static_cast<long long>(s) * per, static_cast<long long>(list.n)));
    const int hi = min(lo + per, list.n);

    // ---- Q as the B operand: head 8 t + g, the columns of this lane's key words ----
    uint32_t qf[NT][W][4];  // 16-bit: 4 words of chunk c + 4 w; 4-bit: nibble pairs of group w, the odd ones / 16
    float q_off[NT][W][2];  // 4-bit: -8 2^-24 sum of the group's q (heads 2c, 2c + 1 of tile t)
    float to_log2[NT][2];   // score of heads 2c, 2c + 1 in base-2 units
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const bool there = 8 * t + g < heads;
        const uint16_t *q = p.q + (bh0 + (there ? 8 * t + g : 0)) * D;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            load_words<4>(qf[t][w], q + (Q4 ? 32 * w + 8 * c : 8 * (c + 4 * w)));
            if (!there) qf[t][w][0] = qf[t][w][1] = qf[t][w][2] = qf[t][w][3] = 0u;
        }
        if constexpr (Q4) {
            // q scaled by a power of two, so that the head's largest |q| is in
            // [2^13, 2^14): fp16 then holds all that matters of either type.
            float x[W][8], mx = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[w][i] = q4::from16<BF16>(static_cast<uint16_t>(qf[t][w][i / 2] >> (16 * (i % 2))));
                    mx = fmaxf(mx, fabsf(x[w][i]));
                }
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
            const int e = min(max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100), 100);
            const float up = __uint_as_float(static_cast<uint32_t>(127 + 13 - e) << 23);
            const float down = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + 11 + e) << 23);  // 2^(24 - 13 + e)
#pragma unroll
            for (int w = 0; w < W; ++w) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // nibble i: column 8 c + i (piece 2c) and 8 c + 4 + i (piece 2c + 1)
                    const float f = i % 2 == 0 ? up : up * 0.0625f;
                    qf[t][w][i] = pack16<false>(x[w][i] * f, x[w][4 + i] * f);
                    const float back = i % 2 == 0 ? 1.f : 16.f;
                    sum += back * (ptx::unpack_lo<false>(qf[t][w][i]) + ptx::unpack_hi<false>(qf[t][w][i]));
                }
                sum += __shfl_xor_sync(kFull, sum, 1);
                sum += __shfl_xor_sync(kFull, sum, 2);
                sum *= -8.f / 16777216.f;
                q_off[t][w][0] = __shfl_sync(kFull, sum, 8 * c);
                q_off[t][w][1] = __shfl_sync(kFull, sum, 8 * c + 4);
            }
            to_log2[t][0] = __shfl_sync(kFull, down, 8 * c);
            to_log2[t][1] = __shfl_sync(kFull, down, 8 * c + 4);
        } else {
            to_log2[t][0] = to_log2[t][1] = p.scale_log2;
        }
    }

    float o[MT][NT][4], m[NT][2], l[NT][2];
    float osum[NT][4];     // 4-bit: row w is the sum of group w's weights
    float r[NT][2][W];     // 4-bit: power-of-two factor of the weights of group w
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) osum[t][i] = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            m[t][k] = -CUDART_INF_F;
            l[t][k] = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) r[t][k][w] = kMostFactor;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[i][t][k] = 0.f;
    }

    Reader<D, Q4> rd{p, list, p.block_table + static_cast<size_t>(b) * p.max_blocks, hk, g, c, false};
    // This warp's i-th tile is list entry lo + warp + 4 i. Lane j holds the
    // pages of its tiles 32 n + j, read a batch ahead.
    const int mine = hi - lo > warp ? (hi - lo - warp + kWarps - 1) / kWarps : 0;
    auto key0_of = [&](int i) { return list.key0(lo + warp + kWarps * i); };
    auto page_of = [&](int i) { return i < mine && p.log2_bs >= 4 ? rd.table[key0_of(i) >> p.log2_bs] : 0; };
    int pages[2] = {page_of(lane), page_of(32 + lane)};
    auto fetch = [&](Tile<D, Q4> &t, int i, int base) {  // base: tile number of pages[0], lane 0
        const int j = i - base;
        const int page = __shfl_sync(kFull, j < 32 ? pages[0] : pages[1], j & 31);
        rd.load(t, key0_of(i), page);
    };

    auto consume = [&](Tile<D, Q4> &t) {
        float ksc[2][W], vsc[2][W];
        if constexpr (Q4) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    ksc[i][w] = q4::from16<BF16>(static_cast<uint16_t>(t.ks[i][w / 2] >> (16 * (w % 2))));
                    vsc[i][w] = q4::from16<BF16>(static_cast<uint16_t>(t.vs[i][w / 2] >> (16 * (w % 2))));
                }
        }
        // ---- S^T = K Q^T ----
        float x[NT][4];
        if constexpr (Q4) {
#pragma unroll
            for (int n = 0; n < NT; ++n) x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                // 16-bit lanes: piece 2c (low) and 2c + 1 (high) of group w
                constexpr int P = D / 64;
                uint32_t a[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    a[i] = __byte_perm(t.k[i][w / 2], t.k[i][P + w / 2], w % 2 == 0 ? 0x5410 : 0x7632);
                const uint32_t a8[2] = {a[0] >> 8, a[1] >> 8};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float acc[4] = {q_off[n][w][0], q_off[n][w][1], q_off[n][w][0], q_off[n][w][1]};
                    mma16816<false>(acc, a[0] & 0x000f000fu, a[1] & 0x000f000fu, a[0] & 0x00f000f0u,
                                    a[1] & 0x00f000f0u, qf[n][w][0], qf[n][w][1]);
                    mma16816<false>(acc, a8[0] & 0x000f000fu, a8[1] & 0x000f000fu, a8[0] & 0x00f000f0u,
                                    a8[1] & 0x00f000f0u, qf[n][w][2], qf[n][w][3]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[n][k] = fmaf(ksc[k / 2][w], acc[k], x[n][k]);
                }
            }
        } else {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        mma16816<kMmaBf16>(x[n], t.k[0][4 * w + 2 * h], t.k[1][4 * w + 2 * h],
                                           t.k[0][4 * w + 2 * h + 1], t.k[1][4 * w + 2 * h + 1], qf[n][w][2 * h],
                                           qf[n][w][2 * h + 1]);
            }
        }
        if (!t.whole) {
            // hidden keys: score -inf, and nothing of their rows is used
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool in = (t.kin >> i) & 1u;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k) x[n][2 * i + k] = in ? x[n][2 * i + k] : -CUDART_INF_F;
                if constexpr (Q4) {
#pragma unroll
                    for (int w = 0; w < W; ++w) vsc[i][w] = in ? vsc[i][w] : 0.f;
                }
            }
            if constexpr (!Q4) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int u = 0; u < S::kVWords; ++u) t.v[i][u] = (t.vin >> i) & 1u ? t.v[i][u] : 0u;
            }
        }
        // ---- weights, maximum moved when a score exceeds it by 2^8 ----
        bool move = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[n][k] *= to_log2[n][k % 2];
                move |= x[n][k] > m[n][k % 2] + kMoveMax;
            }
        if (__any_sync(kFull, move)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float a[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float mx = fmaxf(x[n][k], x[n][2 + k]);
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, off));
                    a[k] = 1.f;
                    if (mx > m[n][k] + kMoveMax) {  // per head: no head's arithmetic depends on another's
                        a[k] = ptx::ex2(m[n][k] - mx);
                        m[n][k] = mx;
                    }
                    l[n][k] *= a[k];
                }
                if constexpr (Q4) {
                    // r takes up the whole powers of two of 1 / a, up to 2^100:
                    // weights stay near 1 and O keeps its size, whatever the
                    // scales of the keys that carry it
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        float f[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            // 2^floor(-log2 a), 1 for a = 1, at most 2^100 (a = 0)
                            const int e = min(126 - static_cast<int>((__float_as_uint(a[k]) - 1u) >> 23), 100);
                            const float up = __uint_as_float(static_cast<uint32_t>(127 + (a[k] > 0.f ? e : 100)) << 23);
                            const float next = fminf(r[n][k][w] * up, kMostFactor);
                            f[k] = a[k] * (next / r[n][k][w]);
                            r[n][k][w] = next;
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int k = 0; k < 4; ++k) o[2 * w + h][n][k] *= f[k % 2];
                        if (g == w) {
                            osum[n][0] *= f[0];
                            osum[n][1] *= f[1];
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int k = 0; k < 4; ++k) o[i][n][k] *= a[k % 2];
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float mk = m[n][k % 2];
                x[n][k] = ptx::ex2(x[n][k] - (mk == -CUDART_INF_F ? 0.f : mk));
                l[n][k % 2] += x[n][k];
            }
        // ---- O^T += V^T P^T ----
        if constexpr (Q4) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint32_t pw[W][2];
                uint32_t most = 0;
#pragma unroll
                for (int w = 0; w < W; ++w)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        pw[w][i] = pack16<false>(x[n][2 * i] * vsc[i][w] * r[n][0][w],
                                                 x[n][2 * i + 1] * vsc[i][w] * r[n][1][w]);
                        most = __vmaxu2(most, pw[w][i]);
                    }
                // weights are >= 0, so their bits order like integers
                const bool again = (most & 0xffffu) > 0x6c00u || (most >> 16) > 0x6c00u;  // 2^12 (a NaN is above)
                if (__any_sync(kFull, again)) {
                    // choose r for each head and group: its largest weight so
                    // far (1 / r, as good as it is known) or in this tile
                    // becomes 1 to 2
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        float f[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float big = fmaxf(x[n][k] * vsc[0][w], x[n][2 + k] * vsc[1][w]);
#pragma unroll
                            for (int off = 4; off < 32; off <<= 1)
                                big = fmaxf(big, __shfl_xor_sync(kFull, big, off));
                            f[k] = 1.f;
                            if (big * r[n][k][w] > kMostWeight) {  // per head and group
                                const int e = min(max(static_cast<int>(__float_as_uint(big) >> 23) - 127, -100), 126);
                                const float next = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                                f[k] = next / r[n][k][w];
                                r[n][k][w] = next;
                            }
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int k = 0; k < 4; ++k) o[2 * w + h][n][k] *= f[k % 2];
                        if (g == w) {
                            osum[n][0] *= f[0];
                            osum[n][1] *= f[1];
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            pw[w][i] = pack16<false>(x[n][2 * i] * vsc[i][w] * r[n][0][w],
                                                     x[n][2 * i + 1] * vsc[i][w] * r[n][1][w]);
                    }
                }
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const uint32_t b0 = transpose8x8(pw[w][0]), b1 = transpose8x8(pw[w][1]);
                    // 16-bit lanes: the even key (low), the odd key (high)
                    const uint32_t sel = w % 2 == 0 ? 0x5410 : 0x7632;
                    const uint32_t v0 = __byte_perm(t.v[0][w / 2], t.v[1][w / 2], sel);
                    const uint32_t v1 = __byte_perm(t.v[2][w / 2], t.v[3][w / 2], sel);
                    mma16816<false>(o[2 * w][n], v0 & 0x000f000fu, v0 & 0x00f000f0u, v1 & 0x000f000fu,
                                    v1 & 0x00f000f0u, b0, b1);
                    const uint32_t y0 = v0 >> 8, y1 = v1 >> 8;
                    mma16816<false>(o[2 * w + 1][n], y0 & 0x000f000fu, y0 & 0x00f000f0u, y1 & 0x000f000fu,
                                    y1 & 0x00f000f0u, b0, b1);
                    const uint32_t one = g == w ? 0x3c003c00u : 0u;  // row w of ones: the weights' sum
                    mma16816<false>(osum[n], one, 0u, one, 0u, b0, b1);
                }
            }
        } else {
            uint32_t b0[NT], b1[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                b0[n] = transpose8x8(pack16<BF16>(x[n][0], x[n][1]));
                b1[n] = transpose8x8(pack16<BF16>(x[n][2], x[n][3]));
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const uint32_t a0 = __byte_perm(t.v[0][i], t.v[1][i], 0x5410);
                const uint32_t a1 = __byte_perm(t.v[0][i], t.v[1][i], 0x7632);
                const uint32_t a2 = __byte_perm(t.v[2][i], t.v[3][i], 0x5410);
                const uint32_t a3 = __byte_perm(t.v[2][i], t.v[3][i], 0x7632);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816<kMmaBf16>(o[i][n], a0, a1, a2, a3, b0[n], b1[n]);
            }
        }
    };

    constexpr int N = S::kDepth;
    Tile<D, Q4> tile[N];
    int base = 0;
#pragma unroll
    for (int d = 0; d < N; ++d)
        if (d < mine) fetch(tile[d], d, base);
    for (int i0 = 0; i0 < mine; i0 += N) {
#pragma unroll
        for (int d = 0; d < N; ++d) {
            const int i = i0 + d;
            if (i < mine) {
                consume(tile[d]);
                if (i + N < mine) fetch(tile[d], i + N, base);
            }
        }
        if (i0 + 2 * N - base >= 32) {  // the first batch of pages is used up
            base += 32;
            pages[0] = pages[1];
            pages[1] = page_of(base + 32 + lane);
        }
    }
    if (rd.bad_page) atomicExch(p.err, kDeviceErrBadIndex);

    // ---- the warps of this partition ----
    __shared__ float sm_m[kWarps][HT], sm_l[kWarps][HT];
    __shared__ __align__(16) float sm_o[kWarps][HT][D];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[t][k] += __shfl_xor_sync(kFull, l[t][k], off);
            if (g == 0) {
                sm_m[warp][8 * t + 2 * c + k] = m[t][k];
                sm_l[warp][8 * t + 2 * c + k] = l[t][k];
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                float lo_v = o[i][t][k], hi_v = o[i][t][2 + k];  // columns col, col + 1
                int col;
                if constexpr (Q4) {
                    const int w = i / 2;
                    const float sum8 = 8.f * __shfl_sync(kFull, osum[t][k], 4 * w + c);
                    const float inv = 1.f / r[t][k][w];
                    lo_v = fmaf(lo_v, 16777216.f, -sum8) * inv;
                    hi_v = fmaf(hi_v, 1048576.f, -sum8) * inv;
                    col = 32 * w + 4 * g + 2 * (i % 2);
                } else {
                    col = 8 * (g + 8 * (i / 4)) + 2 * (i % 4);
                }
                *reinterpret_cast<float2 *>(&sm_o[warp][8 * t + 2 * c + k][col]) = make_float2(lo_v, hi_v);
            }
        }
    }
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
            const size_t at = (bh0 + h) * splits + s;
            *reinterpret_cast<float4 *>(p.o_part + at * D + d) = O;
            if (d == 0) {
                p.m_part[at] = M;
                p.l_part[at] = Lw;
            }
        }
    }
    if (splits == 1) return;

    // ---- the last partition of these heads merges them: a warp per head ----
    __shared__ int is_last;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) is_last = atomicAdd(p.counters + unit, 1) == splits - 1;
    __syncthreads();
    if (!is_last) return;
    __threadfence();
    for (int h = warp; h < heads; h += kWarps) {
        const size_t at = (bh0 + h) * splits;
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

template <int D, bool BF16, bool Q4>
static cudaError_t launch_t(const GqaDecodeParams &p, int B, cudaStream_t st) {
    // one column tile of 8 query heads, or two where a group has more
    const int ht = p.group > 8 ? 16 : 8;
    const unsigned grid = static_cast<unsigned>(B) * p.Hkv * ((p.group + ht - 1) / ht) * p.num_splits;
    if (ht == 8) fa_decode_gqa_kernel<D, BF16, Q4, 1><<<grid, kThreads, 0, st>>>(p);
    else fa_decode_gqa_kernel<D, BF16, Q4, 2><<<grid, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace gqa

int decode_gqa_splits(int sms, int B, int H, int Hkv, int max_keys) {
    const int group = H / Hkv < 1 ? 1 : H / Hkv;
    const long long units = static_cast<long long>(B) * Hkv * ((group + 15) / 16);
    long long s = (3LL * sms + units - 1) / units;  // three CTAs per SM
    const long long most = (static_cast<long long>(max_keys) + 63) / 64;  // at least a 16-key tile for each warp
    s = s < most ? s : most;
    return static_cast<int>(s < 64 ? s : 64);
}

cudaError_t launch_decode_gqa(int D, bool bf16, bool q4, const GqaDecodeParams &p, int B, cudaStream_t st) {
#define FA_GQA(DD, BB, QQ) \
    if (D == DD && bf16 == BB && q4 == QQ) return gqa::launch_t<DD, BB, QQ>(p, B, st);
    FA_GQA(64, false, false) FA_GQA(64, false, true) FA_GQA(64, true, false) FA_GQA(64, true, true)
    FA_GQA(128, false, false) FA_GQA(128, false, true) FA_GQA(128, true, false) FA_GQA(128, true, true)
#undef FA_GQA
    return cudaErrorInvalidValue;
}

}  // namespace fa
