// One-token attention over a paged 16-bit cache with shared key heads, a
// sliding window and sinks (fa_decode_paged_window). The frame (partitions,
// fragments, merge) is that of fa_decode_gqa.cuh.
//
// A warp takes 16 keys at a time, straight from global memory into the
// registers that feed the products (8 KB a tile at D = 128): the next tile's
// keys and values are loaded as soon as the products have taken this one's.
// (Tensor copies into a ring per warp, two tiles ahead, were as fast per byte
// and started later: 55 us against 52 us for 16 sequences of 4100 visible keys
// and 8 key heads, where the bytes alone take 40 us and a launch with nothing to
// read 6 us.)
// Per query head it keeps a running maximum m of the scores in base-2 units
// (moved only when a score exceeds it by 2^8), l = sum 2^(x - m) and
// O = sum 2^(x - m) v; a weight enters the second product as two numbers of the
// cache's type (its rounding and the rest), which costs nothing here; sums are
// fp32. Bound by HBM: K and
// V of the visible keys are read once for a group of up to 16 query heads.
#include <climits>
#include <cmath>

#include "fa.h"
#include "fa_decode_gqa.cuh"

namespace fa {
namespace gqa {

template <int NT>
constexpr int kWindowCtas = NT == 1 ? 3 : 2;  // per SM

template <int D>
struct Tile16 {
    static constexpr int kKWords = D / 8, kVWords = D / 16;
    uint32_t k[2][kKWords];  // keys g, g + 8: chunks (8 columns) c, c + 4, ..
    uint32_t v[4][kVWords];  // keys 2c, 2c + 1, 2c + 8, 2c + 9: chunks g, g + 8
    bool whole;              // every key of the tile is visible (the same for the warp)
    uint32_t kin, vin;       // else: bit i, whether this lane's i-th key row (value row) is
};

template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(kThreads, kWindowCtas<NT>) fa_decode_window_kernel(const GqaDecodeParams p) {
    using T = Tile16<D>;
    constexpr int MT = D / 16, HT = 8 * NT, kRow = 2 * D;
    __shared__ Plan<16, HT> plan;
    __shared__ float sm_m[kWarps][HT], sm_l[kWarps][HT];
    __shared__ __align__(16) float sm_o[kWarps][HT][D];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int g = lane / 4, c = lane % 4;
    plan.make(p);
    for (;;) {
    plan.next(p);
    const Part &job = plan.part;
    if (!job.live) break;
    const KeyList<16> list(p, job.b);
    const int lo = job.lo, hi = min(job.hi, list.n);  // no tile of a sequence without keys
    const int *table = p.block_table + static_cast<size_t>(job.b) * p.max_blocks;

    // ---- this warp's tiles: its i-th is list entry lo + warp + 4 i ----
    const int mine = hi - lo > warp ? (hi - lo - warp + kWarps - 1) / kWarps : 0;
    auto key0_of = [&](int i) { return list.key0(lo + warp + kWarps * i); };
    bool bad_page = false;
    auto page_ok = [&](int page) {
        const bool ok = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_blocks);
        bad_page |= !ok;
        return ok;
    };
    // pages of 16 keys and more: lane j holds the page of tile 32 n + j, two
    // batches, one read ahead
    auto page_of = [&](int i) { return i < mine && p.log2_bs >= 4 ? table[key0_of(i) >> p.log2_bs] : 0; };
    int base = 0;
    int pages0 = page_of(lane), pages1 = page_of(32 + lane);

    auto k_key = [&](int i) { return g + 8 * i; };
    auto v_key = [&](int i) { return 2 * c + (i & 1) + 4 * (i & 2); };
    // address of row `in_page` of this key head in page `page`
    auto row_at = [&](const void *first, unsigned page, unsigned in_page) {
        return static_cast<const char *>(first) +
               static_cast<unsigned long long>(page * p.Hkv + job.hk) * (static_cast<unsigned>(kRow) << p.log2_bs) +
               in_page * kRow;
    };
    auto load_k = [&](T &t, int i, const char *row) {
#pragma unroll
        for (int u = 0; u < T::kKWords / 4; ++u) load_words<4>(&t.k[i][4 * u], row + (c + 4 * u) * 16);
    };
    auto load_v = [&](T &t, int i, const char *row) {
#pragma unroll
        for (int u = 0; u < T::kVWords / 4; ++u) load_words<4>(&t.v[i][4 * u], row + (g + 8 * u) * 16);
    };
    // Tile i. Rows that are not to be read (hidden keys of pages under 16 keys,
    // pages that do not exist) are replaced by others of the cache and masked.
    auto load = [&](T &t, int i) {
        const int key0 = key0_of(i);
        const unsigned mask = (1u << p.log2_bs) - 1;
        t.kin = t.vin = 0;
        if (p.log2_bs >= 4) {
            const int page = __shfl_sync(kFull, i - base < 32 ? pages0 : pages1, i & 31);
            const bool ok = page_ok(page);
            t.whole = ok && key0 >= list.w_lo && key0 + 16 <= list.L;
            if (!t.whole) {
#pragma unroll
                for (int j = 0; j < 2; ++j) t.kin |= (ok && list.sees(key0 + k_key(j)) ? 1u : 0u) << j;
#pragma unroll
                for (int j = 0; j < 4; ++j) t.vin |= (ok && list.sees(key0 + v_key(j)) ? 1u : 0u) << j;
            }
            const unsigned pg = ok ? page : 0;  // 16 rows of page 0 are there to be read (and masked) if not
            const char *kp = row_at(p.k, pg, key0 & mask), *vp = row_at(p.v, pg, key0 & mask);
#pragma unroll
            for (int j = 0; j < 2; ++j) load_k(t, j, kp + k_key(j) * kRow);
#pragma unroll
            for (int j = 0; j < 4; ++j) load_v(t, j, vp + v_key(j) * kRow);
        } else {
            t.whole = false;
            auto row_of = [&](const void *first, int key, uint32_t &in, int bit) {
                bool ok = list.sees(key);
                const int page = ok ? table[key >> p.log2_bs] : 0;
                ok = ok && page_ok(page);
                in |= (ok ? 1u : 0u) << bit;
                return ok ? row_at(first, page, key & mask) : static_cast<const char *>(first);
            };
#pragma unroll
            for (int j = 0; j < 2; ++j) load_k(t, j, row_of(p.k, key0 + k_key(j), t.kin, j));
#pragma unroll
            for (int j = 0; j < 4; ++j) load_v(t, j, row_of(p.v, key0 + v_key(j), t.vin, j));
        }
    };

    // ---- Q as the B operand: head 8 t + g, in the order of the key chunks ----
    uint32_t qf[NT][D / 8];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const bool there = 8 * t + g < job.heads;
        const uint16_t *q = p.q + (job.bh0 + (there ? 8 * t + g : 0)) * D + 8 * c;
#pragma unroll
        for (int u = 0; u < D / 32; ++u) {
            const uint4 v = *reinterpret_cast<const uint4 *>(q + 32 * u);
            qf[t][4 * u] = there ? v.x : 0u;
            qf[t][4 * u + 1] = there ? v.y : 0u;
            qf[t][4 * u + 2] = there ? v.z : 0u;
            qf[t][4 * u + 3] = there ? v.w : 0u;
        }
    }
    float o[MT][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            m[t][k] = kNoMax;
            l[t][k] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[i][t][k] = 0.f;
    }

    T t;
    if (mine > 0) load(t, 0);
    for (int i = 0; i < mine; ++i) {
        // ---- S^T = K Q^T ----
        float x[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
#pragma unroll
            for (int w = 0; w < T::kKWords; w += 2)
                mma16816<BF16>(x[n], t.k[0][w], t.k[1][w], t.k[0][w + 1], t.k[1][w + 1], qf[n][w], qf[n][w + 1]);
        }
        if (!t.whole) {
            // hidden keys: score -inf, and nothing of their rows is used
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const bool in = (t.kin >> j) & 1u;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k) x[n][2 * j + k] = in ? x[n][2 * j + k] : -CUDART_INF_F;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int u = 0; u < T::kVWords; ++u) t.v[j][u] = (t.vin >> j) & 1u ? t.v[j][u] : 0u;
        }
        // ---- weights, maximum moved when a score exceeds it by 2^8 ----
        float e[NT][4];  // exponents x scale - m
        bool move = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                e[n][k] = fmaf(x[n][k], p.scale_log2, -m[n][k % 2]);
                move |= e[n][k] > kMoveMax;
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
                    if (fmaf(mx, p.scale_log2, -m[n][k]) > kMoveMax) {  // per head: no head depends on another
                        const float next = mx * p.scale_log2;
                        a[k] = ptx::ex2(m[n][k] - next);
                        m[n][k] = next;
                    }
                    l[n][k] *= a[k];
                }
#pragma unroll
                for (int j = 0; j < MT; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[j][n][k] *= a[k % 2];
#pragma unroll
                for (int k = 0; k < 4; ++k) e[n][k] = fmaf(x[n][k], p.scale_log2, -m[n][k % 2]);
            }
        }
        uint32_t b0[NT], b1[NT], r0[NT], r1[NT];  // weights, and what their rounding leaves
        auto rest = [](uint32_t w, float lo, float hi) {
            return pack16<BF16>(lo - ptx::unpack_lo<BF16>(w), hi - ptx::unpack_hi<BF16>(w));
        };
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[n][k] = ptx::ex2(e[n][k]);
                l[n][k % 2] += x[n][k];
            }
            const uint32_t w0 = pack16<BF16>(x[n][0], x[n][1]), w1 = pack16<BF16>(x[n][2], x[n][3]);
            b0[n] = transpose8x8(w0);
            b1[n] = transpose8x8(w1);
            r0[n] = transpose8x8(rest(w0, x[n][0], x[n][1]));
            r1[n] = transpose8x8(rest(w1, x[n][2], x[n][3]));
        }
        // ---- O^T += V^T P^T ----
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const uint32_t a0 = __byte_perm(t.v[0][j], t.v[1][j], 0x5410);
            const uint32_t a1 = __byte_perm(t.v[0][j], t.v[1][j], 0x7632);
            const uint32_t a2 = __byte_perm(t.v[2][j], t.v[3][j], 0x5410);
            const uint32_t a3 = __byte_perm(t.v[2][j], t.v[3][j], 0x7632);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma16816<BF16>(o[j][n], a0, a1, a2, a3, b0[n], b1[n]);
                mma16816<BF16>(o[j][n], a0, a1, a2, a3, r0[n], r1[n]);
            }
        }
        if (i + 1 - base >= 32) {
            base += 32;
            pages0 = pages1;
            pages1 = page_of(base + 32 + lane);
        }
        if (i + 1 < mine) load(t, i + 1);
    }
    if (bad_page) atomicExch(p.err, kDeviceErrBadIndex);

#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[n][k] += __shfl_xor_sync(kFull, l[n][k], off);
            const int head = 8 * n + 2 * c + k;
            if (g == 0) {
                sm_m[warp][head] = m[n][k] == kNoMax ? -CUDART_INF_F : m[n][k];
                sm_l[warp][head] = l[n][k];
            }
#pragma unroll
            for (int j = 0; j < MT; ++j)
                *reinterpret_cast<float2 *>(&sm_o[warp][head][8 * (g + 8 * (j / 4)) + 2 * (j % 4)]) =
                    make_float2(o[j][n][k], o[j][n][2 + k]);
        }
    merge<D, BF16, HT>(p, job, sm_m, sm_l, sm_o);
    }
}

template <int D, bool BF16, int NT>
static cudaError_t launch_t(GqaDecodeParams p, int sms, cudaStream_t st) {
    const unsigned grid = decode_gqa_grid(p, sms, kWindowCtas<NT>, 8 * NT);
    fa_decode_window_kernel<D, BF16, NT><<<grid, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace gqa

// Whether the balanced plan serves: the tables hold more than 32 tiles of 16
// keys for each CTA of a wave (the plan costs a CTA about 2 us), and all tiles
// can be counted in 32 bits.
static bool gqa_balanced(long long units, long long keys, long long wave) {
    const long long tiles = units * (keys / 16 + 2);
    return tiles > 32 * wave && units * (keys / 16 + 16) <= INT_MAX;
}

int decode_gqa_splits(int sms, int B, int H, int Hkv, int max_keys) {
    const int group = H / Hkv < 1 ? 1 : H / Hkv;
    const long long units = static_cast<long long>(B) * Hkv * ((group + 15) / 16);
    const long long wave = 3LL * sms;
    // Little work: one wave of CTAs, none with fewer than 256 keys (joining
    // parts costs 4 us, a second wave as much again). More: the balanced plan,
    // which cuts the longest sequence into as many parts as its share of the
    // batch asks for, and two more for parts that straddle units.
    const long long plain = wave / units > 1 ? wave / units : 1, keys = (static_cast<long long>(max_keys) + 255) / 256;
    const long long balanced = 8LL * sms / units + 3;
    const long long s = gqa_balanced(units, max_keys, wave) ? balanced : (plain < keys ? plain : keys);
    // Parts are read side by side and joined by one CTA (0.14, 0.25 and 0.54 us
    // each for 1, 8 and 16 heads), so few units do best with a number that grows
    // as the square root of their keys: 64 up to 131072 of them. (One key head, 8
    // query heads, D = 128, us over 16-bit pages / the 4-bit cache with 32, 64, 96,
    // 152, 192, 256 and 456 parts: 16384 keys 29/29, 33/35, 39/41, 52/53, 64/64,
    // 78/78, 133/133; 131072: 90/64, 64/55, 61/59, 68/67, 76/78, 89/89, 141/139; 2^20:
    // 620/297, 330/174, 240/141, 186/125, 176/133, 173/137, 208/176.)
    const long long most = max_keys > 131072 ? static_cast<long long>(64 * std::sqrt(max_keys / 131072.0)) : 64;
    const long long cap = most < FA_MAX_SPLITS ? most : FA_MAX_SPLITS;
    return static_cast<int>(s < cap ? s : cap);
}

unsigned decode_gqa_grid(GqaDecodeParams &p, int sms, int ctas_per_sm, int heads_per_unit) {
    const long long units = static_cast<long long>(p.B) * p.Hkv * ((p.group + heads_per_unit - 1) / heads_per_unit);
    const long long all = units * p.num_splits, wave = static_cast<long long>(sms) * ctas_per_sm;
    const long long cap = static_cast<long long>(p.max_blocks) << p.log2_bs;
    const long long seen = p.window > 0 && static_cast<long long>(p.window) + p.sinks < cap ? p.window + p.sinks : cap;
    p.balanced = p.num_splits > 1 && p.B <= gqa::kPlanSeqs && gqa_balanced(units, seen, wave);
    return static_cast<unsigned>(p.balanced && wave < all ? wave : all);
}

cudaError_t launch_decode_window(int D, bool bf16, const GqaDecodeParams &p, int sms, cudaStream_t st) {
    // one column tile of 8 query heads, or two where a group has more
    const int NT = p.group > 8 ? 2 : 1;
#define FA_GQA(DD, BB, NN) \
    if (D == DD && bf16 == BB && NT == NN) return gqa::launch_t<DD, BB, NN>(p, sms, st);
    FA_GQA(64, false, 1) FA_GQA(64, false, 2) FA_GQA(64, true, 1) FA_GQA(64, true, 2)
    FA_GQA(128, false, 1) FA_GQA(128, false, 2) FA_GQA(128, true, 1) FA_GQA(128, true, 2)
#undef FA_GQA
    return cudaErrorInvalidValue;
}

}  // namespace fa
