// One-token attention over the paged 4-bit cache (fa_decode_paged_q4). The
// frame (partitions, fragments, merge) is that of fa_decode_gqa.cuh.
//
// Mathematics. A warp keeps, per query head, a running maximum m of the scores
// x_j in base-2 units, l = sum_j 2^(x_j - m) and O = sum_j 2^(x_j - m) v_j over
// its keys; m is moved only when a score exceeds it by 2^8. The cache holds
// k = s (u - 8), u a nibble, s per 32 columns w, so
//   x = scale log2(e) sum_w s_w (sum_d q_d u_d - 8 sum_d q_d),
//   O = sum_j (p_j s_j) (u_j - 8).
// A nibble is a number as it stands: masked out of its word, nibble 0 of a
// 16-bit lane is the fp16 number u 2^-24 and nibble 1 is u 2^-20 (below the
// normal numbers, which the tensor core takes exactly), so two values cost one
// logical operation. The factor 16 goes into q (keys) or stays in the rows of
// O (values); the 8 is where the sum starts (keys: the term is the same for
// all of them) or goes off pairs of values by one fp16 subtraction, exactly
// (values: each key has its weight, and no digits are lost to 8 sum p s). The
// weights p_j s_j are rounded to fp16 (11 bits, for either type of cache)
// after a power-of-two factor r per head and column group that keeps the
// largest of them between 2^-4 and 2 whatever the scales (a move of m may halve
// it: weights 2^-20 of the largest keep few bits); products exact, sums fp32.
//
// What bounds it: HBM wants 24 bytes (48 values) per SM and cycle, so the few
// instructions a value costs fill the issue slots; everything above is there
// to save instructions. Tiles of 32 keys come by asynchronous copies into a
// ring per warp (4.5 KB a tile at D = 128, two in flight), which leaves the
// registers to the accumulators: four CTAs (16 warps) per SM. 16 sequences of
// 16384 to 32768 keys, 8 key heads, 32 heads, D = 128: 113 us, 4.2 TB/s, where
// the bytes alone take 70 us; some 324 warp instructions per 16 keys, the ALU
// pipe half of the time. (Bulk copies in place of these, eight per tile with 16-key
// pages, cost a loop over the issuing lanes each and 8 us of it.)
#include "fa_decode_gqa.cuh"

namespace fa {
namespace gqa {

// 16 bytes from global to shared memory, in this thread's current copy group.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>  // wait until all but the newest N groups have landed
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr float kMostWeight = 2.f;  // weights of this size and more choose their factor r again
constexpr float kMostFactor = 1.2676506002282294e30f;  // 2^100: r before any weight is known

template <int D, int NT>
struct Q4Shape {
    static constexpr int kTile = 32;               // keys per ring stage
    static constexpr int kW = D / 32;              // column groups
    static constexpr int kRow = D / 2, kSRow = D / 16;   // bytes of a row's codes, of its scales
    static constexpr int kKWords = D / 32, kVWords = D / 64, kSWords = D / 64;
    static constexpr int kMTiles = D / 16;         // 16-column tiles of O^T
    static constexpr int kStages = 256 / D;         // four CTAs fit an SM
    static constexpr int kV = kTile * kRow, kKS = 2 * kV, kVS = kKS + kTile * kSRow;  // offsets in a stage
    static constexpr int kStageBytes = kVS + kTile * kSRow;
    static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
    static constexpr int kMergeBytes = kWarps * 8 * NT * D * 4;
    // offsets of the stages' visible keys, of Q's fragments and of -8 sum q as
    // accumulators ([NT][kW][32 lanes][4 words])
    static constexpr int kSeen = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;
    static constexpr int kQ = kSeen + kWarps * kStages * 4, kQSum = kQ + NT * kW * 512;
    static constexpr int kSmemBytes = kQSum + NT * kW * 512;
    static constexpr int kCtas = NT == 1 ? 4 : 2;  // per SM
};

// The code pairs of a word (two 16-bit lanes of four nibbles each): nibbles 0
// and 2 as fp16 numbers u 2^-24, 1 and 3 as u 2^-20.
__device__ __forceinline__ void unpack_codes(uint32_t x, uint32_t (&out)[4]) {
    const uint32_t y = x >> 8;
    out[0] = x & 0x000f000fu;
    out[1] = x & 0x00f000f0u;
    out[2] = y & 0x000f000fu;
    out[3] = y & 0x00f000f0u;
}
// ... less 8.
__device__ __forceinline__ void minus8(uint32_t (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = sub16x2(x[i], i % 2 == 0 ? 0x00080008u : 0x00800080u);
}
constexpr uint32_t kMinus8Lo = 0x80088008u;  // fp16 pair -8 2^-24
constexpr uint32_t kMinus8Hi = 0x80808080u;  // fp16 pair -8 2^-20

template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(kThreads, (Q4Shape<D, NT>::kCtas)) fa_decode_q4_kernel(const GqaDecodeParams p) {
    using S = Q4Shape<D, NT>;
    constexpr int W = S::kW, MT = S::kMTiles, HT = 8 * NT;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Plan<S::kTile, HT> plan;
    __shared__ float sm_m[kWarps][HT], sm_l[kWarps][HT];
    auto sm_o = reinterpret_cast<float (*)[HT][D]>(smem);  // over the rings, once every warp is done with its own
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int g = lane / 4, c = lane % 4;
    const bool ring = p.log2_bs >= 4;  // 16 keys of a page follow one another
    uint8_t *const my_ring = smem + warp * S::kStages * S::kStageBytes;
    const uint32_t stage0 = ptx::smem_addr(my_ring);
    const uint32_t seen_at = ptx::smem_addr(smem) + S::kSeen + warp * S::kStages * 4;
    const unsigned page_mask = (1u << p.log2_bs) - 1;
    plan.make(p);
    for (;;) {
    plan.next(p);
    const Part &job = plan.part;
    if (!job.live) break;
    const KeyList<S::kTile> list(p, job.b);
    const int lo = job.lo, hi = min(job.hi, list.n);  // no tile of a sequence without keys
    const int *table = p.block_table + static_cast<size_t>(job.b) * p.max_blocks;

    // ---- this warp's tiles: its i-th is list entry lo + warp + 4 i ----
    const int mine = hi - lo > warp ? (hi - lo - warp + kWarps - 1) / kWarps : 0;
    auto key0_of = [&](int i) { return list.key0(lo + warp + kWarps * i); };
    bool bad_page = false;
    // Lane j holds where keys 16 (j % 2) .. + 15 of tile 16 n + j / 2 are, in
    // units of 16 rows (they fit 32 bits), or kNone (no visible key there, or no
    // such page); two batches, one read ahead.
    constexpr unsigned kNone = 0xffffffffu;
    auto place_of = [&](int i) {
        if (!ring || i >= mine) return kNone;
        const int key = key0_of(i) + 16 * (lane & 1);
        if (!list.sees16(key)) return kNone;
        const int page = table[key >> p.log2_bs];
        const bool ok = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_blocks);
        bad_page |= !ok;
        if (!ok) return kNone;
        return ((static_cast<unsigned>(page) * p.Hkv + job.hk) << (p.log2_bs - 4)) + ((key & page_mask) >> 4);
    };
    int base = 0;  // tile of places0, lane 0
    unsigned places0 = place_of(lane / 2), places1 = place_of(16 + lane / 2);

    // ---- asynchronous copies, 16 bytes a lane: 16 keys' codes are 16 kRow
    // bytes in a row of each array, their scales 16 kSRow bytes ----
    const bool v_scales = lane >= 16;  // the scales: half a warp each
    const bool scale_lane = (lane & 15) < S::kSRow;
    const char *const scale_base = static_cast<const char *>(v_scales ? p.vs : p.ks) + 16 * (lane & 15);
    const uint32_t scale_dst = stage0 + (v_scales ? S::kVS : S::kKS) + 16 * (lane & 15);
    const char *const k_base = static_cast<const char *>(p.k) + 16 * lane;
    const char *const v_base = static_cast<const char *>(p.v) + 16 * lane;
    auto copy_half = [&](int half, unsigned place, uint32_t at) {
        const unsigned long long codes = static_cast<unsigned long long>(place) * (16 * S::kRow);
        const char *k = k_base + codes, *v = v_base + codes;
#pragma unroll
        for (int j = 0; j < 16 * S::kRow / 512; ++j) {
            copy16(at + half * 16 * S::kRow + 512 * j + 16 * lane, k + 512 * j);
            copy16(at + S::kV + half * 16 * S::kRow + 512 * j + 16 * lane, v + 512 * j);
        }
        if (scale_lane)
            copy16(scale_dst + (at - stage0) + half * 16 * S::kSRow,
                   scale_base + static_cast<unsigned long long>(place) * (16 * S::kSRow));
    };
    // Tiles are started in order, one copy group each (empty past the last).
    // Leaves the tile's visible keys with its stage.
    auto start = [&](int i, int stage) {
        if (i < mine) {
            if (i - base == 16) {
                base += 16;
                places0 = places1;
                places1 = place_of(base + 16 + lane / 2);
            }
            const int key0 = key0_of(i);
            const unsigned a = __shfl_sync(kFull, places0, 2 * (i & 15)),
                           b = __shfl_sync(kFull, places0, 2 * (i & 15) + 1);
            uint32_t seen = kFull;
            if (a == kNone || b == kNone || key0 < list.w_lo || key0 + 32 > list.L)
                seen = __ballot_sync(kFull, (lane < 16 ? a : b) != kNone && list.sees(key0 + lane));
            if (lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(seen_at + 4 * stage), "r"(seen) : "memory");
            const uint32_t at = stage0 + stage * S::kStageBytes;
            if (a != kNone) copy_half(0, a, at);
            if (b != kNone) copy_half(1, b, at);
        }
        copy_commit();
    };
    // Pages of fewer than 16 keys: a lane copies one key's rows by itself.
    // Returns the tile's visible keys.
    auto copy_rows = [&](int key0) -> uint32_t {
        const int key = key0 + lane;
        bool ok = list.sees(key);
        if (ok) {
            const int page = table[key >> p.log2_bs];
            ok = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_blocks);
            bad_page |= !ok;
            if (ok) {
                const size_t row = ((static_cast<size_t>(page) * p.Hkv + job.hk) << p.log2_bs) +
                                   (key & ((1 << p.log2_bs) - 1));
                uint8_t *dst = my_ring;
                const uint4 *k = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.k) + row * S::kRow);
                const uint4 *v = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.v) + row * S::kRow);
#pragma unroll
                for (int j = 0; j < S::kRow / 16; ++j) {
                    reinterpret_cast<uint4 *>(dst + lane * S::kRow)[j] = k[j];
                    reinterpret_cast<uint4 *>(dst + S::kV + lane * S::kRow)[j] = v[j];
                }
#pragma unroll
                for (int j = 0; j < S::kSWords; ++j) {
                    reinterpret_cast<uint32_t *>(dst + S::kKS + lane * S::kSRow)[j] =
                        static_cast<const uint32_t *>(p.ks)[row * S::kSWords + j];
                    reinterpret_cast<uint32_t *>(dst + S::kVS + lane * S::kSRow)[j] =
                        static_cast<const uint32_t *>(p.vs)[row * S::kSWords + j];
                }
            }
        }
        const uint32_t seen = __ballot_sync(kFull, ok);
        __syncwarp();
        return seen;
    };
    if (ring)
        for (int i = 0; i < S::kStages; ++i) start(i, i);

    // ---- Q as the B operand: head 8 t + g, in the order of the key words
    // (nibble pairs of group w; the odd ones' q / 16); in shared memory, the
    // registers hold the accumulators ----
    const uint32_t q_at = ptx::smem_addr(smem) + S::kQ + 16 * lane;
    float to_log2[NT][2];   // of heads 2c, 2c + 1: what turns a sum into a score in base-2 units
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const bool there = 8 * t + g < job.heads;
        const uint16_t *q = p.q + (job.bh0 + (there ? 8 * t + g : 0)) * D + 8 * c;
        // q scaled by a power of two, so that the head's largest |q| is in
        // [2^13, 2^14): fp16 then holds all that matters of either type
        float x[W][8], mx = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const uint4 v = *reinterpret_cast<const uint4 *>(q + 32 * w);
            const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[w][i] = there ? q4::from16<BF16>(static_cast<uint16_t>(word[i / 2] >> (16 * (i % 2)))) : 0.f;
                mx = fmaxf(mx, fabsf(x[w][i]));
            }
        }
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
        const int e = min(max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100), 100);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 13 - e) << 23);
        const float down = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + 11 + e) << 23);  // 2^(24 - 13 + e)
#pragma unroll
        for (int w = 0; w < W; ++w) {
            uint32_t f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // nibble i: column 8 c + i (piece 2c) and 8 c + 4 + i (piece 2c + 1)
                const float by = i % 2 == 0 ? up : up * 0.0625f;
                f[i] = pack16<false>(x[w][i] * by, x[w][4 + i] * by);
            }
            // -8 sum_d q_d of the group, where the product of a tile starts
            float acc[4];
            mma16816<false>(acc, kMinus8Lo, kMinus8Lo, kMinus8Hi, kMinus8Hi, f[0], f[1], 0.f, 0.f, 0.f, 0.f);
            mma16816<false>(acc, kMinus8Lo, kMinus8Lo, kMinus8Hi, kMinus8Hi, f[2], f[3]);
            if (warp == 0) {  // every warp has the same: one writes
                *reinterpret_cast<uint4 *>(smem + S::kQ + (t * W + w) * 512 + 16 * lane) =
                    make_uint4(f[0], f[1], f[2], f[3]);
                *reinterpret_cast<float4 *>(smem + S::kQSum + (t * W + w) * 512 + 16 * lane) =
                    make_float4(acc[0], acc[1], acc[2], acc[3]);
            }
        }
        to_log2[t][0] = __shfl_sync(kFull, down, 8 * c);
        to_log2[t][1] = __shfl_sync(kFull, down, 8 * c + 4);
    }

    __syncthreads();
    float o[MT][NT][4], nm[NT][2], l[NT][2];  // nm: -m, as the exponents take it
    float r[NT][W][2];  // power-of-two factor of the weights of group w
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            nm[t][k] = -kNoMax;
            l[t][k] = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) r[t][w][k] = kMostFactor;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[i][t][k] = 0.f;
    }

    // Which key stands in which row of the products is free: rows 2 and 3, and
    // 6 and 7, change places, so that the value rows of one access fall on all
    // shared-memory banks.
    auto row_key = [](int row) { return row ^ ((row >> 1) & 1); };

    // One tile at `stage`; bit k of `seen`: key0 + k is visible.
    auto consume = [&](uint32_t stage, uint32_t seen) {
        // ---- S^T = K Q^T, 16 keys at a time ----
        float x[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t k[2][S::kKWords], ks[2][S::kSWords];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = 16 * h + 8 * i + row_key(g);
                shared_words<S::kKWords>(k[i], stage + row * S::kRow + c * (D / 8));
                shared_words<S::kSWords>(ks[i], stage + S::kKS + row * S::kSRow);
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
                uint32_t a[2][4];
                float sc[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // 16-bit lanes: piece 2c (low) and 2c + 1 (high) of group w
                    unpack_codes(__byte_perm(k[i][w / 2], k[i][D / 64 + w / 2], w % 2 == 0 ? 0x5410 : 0x7632), a[i]);
                    sc[i] = q4::from16<BF16>(static_cast<uint16_t>(ks[i][w / 2] >> (16 * (w % 2))));
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    uint32_t q[4];
                    shared_words<4>(q, q_at + (n * W + w) * 512);
                    uint32_t start_at[4];
                    shared_words<4>(start_at, q_at + S::kQSum - S::kQ + (n * W + w) * 512);
                    float acc[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[j] = __uint_as_float(start_at[j]);
                    mma16816<false>(acc, a[0][0], a[1][0], a[0][1], a[1][1], q[0], q[1]);
                    mma16816<false>(acc, a[0][2], a[1][2], a[0][3], a[1][3], q[2], q[3]);
#pragma unroll
                    for (int j = 0; j < 4; j += 2) {
                        const uint64_t s2 = ptx::pk2(sc[j / 2], sc[j / 2]), y = ptx::pk2(acc[j], acc[j + 1]);
                        ptx::upk2(w == 0 ? ptx::fmul2(s2, y) : ptx::ffma2(s2, y, ptx::pk2(x[h][n][j], x[h][n][j + 1])),
                                  x[h][n][j], x[h][n][j + 1]);
                    }
                }
            }
        }
        const bool whole = seen == kFull;
        if (!whole) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool in = (seen >> (16 * h + 8 * i + row_key(g))) & 1u;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int k = 0; k < 2; ++k) x[h][n][2 * i + k] = in ? x[h][n][2 * i + k] : -CUDART_INF_F;
                }
        }
        // ---- weights, maximum moved when a score exceeds it by 2^8 ----
        float e[2][NT][4];  // exponents x to_log2 - m
        float most_e[NT];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 4; k += 2)
                    ptx::upk2(ptx::ffma2(ptx::pk2(x[h][n][k], x[h][n][k + 1]), ptx::pk2(to_log2[n][0], to_log2[n][1]),
                                         ptx::pk2(nm[n][0], nm[n][1])),
                              e[h][n][k], e[h][n][k + 1]);
#pragma unroll
        for (int n = 0; n < NT; ++n)
            most_e[n] = fmaxf(ptx::fmax3(ptx::fmax3(e[0][n][0], e[0][n][1], e[0][n][2]),
                                         ptx::fmax3(e[0][n][3], e[1][n][0], e[1][n][1]), e[1][n][2]), e[1][n][3]);
        if (__any_sync(kFull, (NT == 1 ? most_e[0] : fmaxf(most_e[0], most_e[NT - 1])) > kMoveMax)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float a[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float mx = fmaxf(fmaxf(x[0][n][k], x[0][n][2 + k]), fmaxf(x[1][n][k], x[1][n][2 + k]));
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, off));
                    a[k] = 1.f;
                    if (fmaf(mx, to_log2[n][k], nm[n][k]) > kMoveMax) {  // per head: no head depends on another
                        const float next = mx * to_log2[n][k];
                        a[k] = ptx::ex2(-nm[n][k] - next);
                        nm[n][k] = -next;
                    }
                    l[n][k] *= a[k];
                }
                // r takes up the whole powers of two of 1 / a, up to 2^100:
                // weights stay near 1 and O keeps its size, whatever the scales
                // of the keys that carry it
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    float f[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        // 2^floor(-log2 a), 1 for a = 1, at most 2^100 (a = 0)
                        const int ex = min(126 - static_cast<int>((__float_as_uint(a[k]) - 1u) >> 23), 100);
                        const float up = __uint_as_float(static_cast<uint32_t>(127 + (a[k] > 0.f ? ex : 100)) << 23);
                        const float next = fminf(r[n][w][k] * up, kMostFactor);
                        f[k] = a[k] * (next / r[n][w][k]);
                        r[n][w][k] = next;
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int k = 0; k < 4; ++k) o[2 * w + i][n][k] *= f[k % 2];
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) e[h][n][k] = fmaf(x[h][n][k], to_log2[n][k % 2], nm[n][k % 2]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    x[h][n][k] = ptx::ex2(e[h][n][k]);
                    x[h][n][k + 1] = ptx::ex2(e[h][n][k + 1]);
                    ptx::upk2(ptx::fadd2(ptx::pk2(l[n][0], l[n][1]), ptx::pk2(x[h][n][k], x[h][n][k + 1])), l[n][0],
                              l[n][1]);
                }
        // ---- O^T += V^T P^T, 16 keys at a time ----
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t vs[2][S::kSWords];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = 16 * h + 8 * i + row_key(g);
                shared_words<S::kSWords>(vs[i], stage + S::kVS + row * S::kSRow);
            }
            if (!whole) {  // nothing of a hidden key is used
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (!((seen >> (16 * h + 8 * i + row_key(g))) & 1u))
#pragma unroll
                        for (int j = 0; j < S::kSWords; ++j) vs[i][j] = 0u;
            }
            auto v_scale = [&](int i, int w) {
                return q4::from16<BF16>(static_cast<uint16_t>(vs[i][w / 2] >> (16 * (w % 2))));
            };
            uint32_t pw[NT][W][2];
            auto weights = [&](int n, int w) {
                const uint64_t rr = ptx::pk2(r[n][w][0], r[n][w][1]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float s = v_scale(i, w);
                    const uint64_t y = ptx::fmul2(ptx::fmul2(ptx::pk2(x[h][n][2 * i], x[h][n][2 * i + 1]), ptx::pk2(s, s)), rr);
                    float y0, y1;
                    ptx::upk2(y, y0, y1);
                    pw[n][w][i] = pack16<false>(y0, y1);
                }
            };
            uint32_t most = 0;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    weights(n, w);
                    most |= pw[n][w][0] | pw[n][w][1];
                }
            // the weights are >= 0: bit 14 of an fp16 number says that it is 2 or more
            if (__any_sync(kFull, (most & 0x40004000u) != 0u)) {
                // choose r for each head and group whose weights grew out of
                // it: the largest of these keys' becomes 1/16 to 1/8
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        float f[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float big = fmaxf(x[h][n][k] * v_scale(0, w), x[h][n][2 + k] * v_scale(1, w));
#pragma unroll
                            for (int off = 4; off < 32; off <<= 1) big = fmaxf(big, __shfl_xor_sync(kFull, big, off));
                            f[k] = 1.f;
                            if (big * r[n][w][k] >= kMostWeight * 0.999f) {  // per head and group
                                const int ex = min(max(static_cast<int>(__float_as_uint(big) >> 23) - 123, -100), 126);
                                const float next = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
                                f[k] = next / r[n][w][k];
                                r[n][w][k] = next;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int k = 0; k < 4; ++k) o[2 * w + i][n][k] *= f[k % 2];
                        weights(n, w);
                    }
            }
            uint32_t v[4][S::kVWords];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 16 * h + 8 * (i >> 1) + row_key(2 * c + (i & 1));
                shared_words<S::kVWords>(v[i], stage + S::kV + row * S::kRow + g * S::kSRow);
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
                // 16-bit lanes: the even row (low), the odd row (high)
                const uint32_t sel = w % 2 == 0 ? 0x5410 : 0x7632;
                uint32_t a0[4], a1[4];
                unpack_codes(__byte_perm(v[0][w / 2], v[1][w / 2], sel), a0);
                unpack_codes(__byte_perm(v[2][w / 2], v[3][w / 2], sel), a1);
                minus8(a0);
                minus8(a1);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint32_t b0 = transpose8x8(pw[n][w][0]), b1 = transpose8x8(pw[n][w][1]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        mma16816<false>(o[2 * w + i][n], a0[2 * i], a0[2 * i + 1], a1[2 * i], a1[2 * i + 1], b0, b1);
                    }
                }
            }
        }
    };

    if (ring) {
        int st = 0;
        for (int i = 0; i < mine; ++i) {
            copy_wait<S::kStages - 1>();  // this lane's copies of tile i, and all lanes' after the barrier
            __syncwarp();
            uint32_t seen;
            shared_words<1>(&seen, seen_at + 4 * st);
            consume(stage0 + st * S::kStageBytes, seen);
            __syncwarp();  // the stage is read: it may be filled again
            start(i + S::kStages, st);
            st = st + 1 == S::kStages ? 0 : st + 1;
        }
    } else {
        for (int i = 0; i < mine; ++i) {
            const uint32_t seen = copy_rows(key0_of(i));
            consume(stage0, seen);
            __syncwarp();
        }
    }
    if (bad_page) atomicExch(p.err, kDeviceErrBadIndex);

    __syncthreads();  // every warp is done with its ring
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[t][k] += __shfl_xor_sync(kFull, l[t][k], off);
            const int head = 8 * t + 2 * c + k;
            if (g == 0) {
                sm_m[warp][head] = nm[t][k] == -kNoMax ? -CUDART_INF_F : -nm[t][k];
                sm_l[warp][head] = l[t][k];
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float inv = 1.f / r[t][w][k];  // a power of two
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<float2 *>(&sm_o[warp][head][32 * w + 4 * g + 2 * i]) =
                        make_float2(o[2 * w + i][t][k] * 16777216.f * inv, o[2 * w + i][t][2 + k] * 1048576.f * inv);
            }
        }
    merge<D, BF16, HT>(p, job, sm_m, sm_l, sm_o);
    __syncthreads();  // sm_o is read: the next part's copies go there
    }
}

template <int D, bool BF16, int NT>
static cudaError_t launch_t(GqaDecodeParams p, int sms, cudaStream_t st) {
    using S = Q4Shape<D, NT>;
    auto kern = fa_decode_q4_kernel<D, BF16, NT>;
    const unsigned grid = decode_gqa_grid(p, sms, S::kCtas, 8 * NT);
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kern), S::kSmemBytes, done);
    if (e != cudaSuccess) return e;
    kern<<<grid, kThreads, S::kSmemBytes, st>>>(p);
    return cudaGetLastError();
}

}  // namespace gqa

cudaError_t launch_decode_q4(int D, bool bf16, const GqaDecodeParams &p, int sms, cudaStream_t st) {
    // one column tile of 8 query heads, or two where a group has more
    const int NT = p.group > 8 ? 2 : 1;
#define FA_Q4(DD, BB, NN) \
    if (D == DD && bf16 == BB && NT == NN) return gqa::launch_t<DD, BB, NN>(p, sms, st);
    FA_Q4(64, false, 1) FA_Q4(64, false, 2) FA_Q4(64, true, 1) FA_Q4(64, true, 2)
    FA_Q4(128, false, 1) FA_Q4(128, false, 2) FA_Q4(128, true, 1) FA_Q4(128, true, 2)
#undef FA_Q4
    return cudaErrorInvalidValue;
}

}  // namespace fa
