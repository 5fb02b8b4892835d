// The attention weight that each key of a paged cache receives from a chunk of
// queries (fa_kv_weights): w[b, hk, j] += sum over the chunk's queries i that see
// key j and the query heads g of key head hk of exp(scale q_ig . k_j - lse_ig),
// the softmax weights of the attention that gave lse.
//
// S^T = K Q^T on the tensor core, keys down the TMEM lanes: a thread owns a key
// and sums its row, so the sums need no exchange, no atomics, and come in one
// order. A unit is two key tiles of one key head, which stay in shared memory
// while the query tiles that see any of them stream past (rows as in
// fa_chunk.cuh); with one key tile, queries would come from L2 at 64 bytes a clock
// and SM, twice what it gives. Two warpgroups take the steps in turn, each with a
// TMEM buffer of 128 columns for each key tile: one waits for its scores while the
// other keeps the exponentials going. -lse log2 e of a step's columns comes through
// shared memory, -inf where a column is no query.
//
// Only the warps that load walk the units; the others are told of a step by what
// the -lse ring holds beside it. A kernel whose twelve warps all walked them was bound
// by its instruction cache where units are short (one token: 19 % of fetches missed it).
//
// Bound: single tokens by reading the keys (16 sequences of 4100 to 8192 keys, 8 key
// heads, D = 128: 40 us, 5.2 TB/s, of which some 8 us are the launch and the way to the
// first keys; of 32000 keys 177 us, 6.0 TB/s, with 128-key pages 6.4). Long chunks by
// the exponentials: 512 tokens of four sequences of 8704 to 16896 keys, 32 heads on 8,
// take 207 us, 1205 TFLOP/s, 53 % of the rate of ex2; without the products 204, products
// and loads alone 169 (both operands come from shared memory).
// Measured beside this: both warpgroups on every step, half of the columns each, 229;
// a step's scores loaded while the step before is added up, 265 to 317; sums two at a
// time 248; four warpgroups 225. For single tokens: query tiles of 32 rows and three
// units of keys in flight 43, pages looked up a unit ahead 40 (29 -> 31 at D = 64).
#include "fa_paged.cuh"

namespace fa {
namespace weights {

using namespace paged;

constexpr int kThreads = 384;
constexpr int kUnitKeys = 2 * kBlockN;
constexpr int kStart = 1;  // what a unit's start costs, in query tiles

template <int D>
struct Shape {
    static constexpr int kColBlocks = D / 64;
    static constexpr int kBlockBytes = FwdShape<D>::kBlockBytes;
    static constexpr int kTileBytes = FwdShape<D>::kTileBytes;
    static constexpr int kKUnits = D == 128 ? 2 : 4;   // units whose keys are loaded or loading
    static constexpr int kQStages = D == 128 ? 3 : 4;
    static constexpr int kLStages = 3, kLBytes = 512 + 32;  // -lse log2 e of 128 columns, and the step's Step
    static constexpr int kOffK = 0;
    static constexpr int kOffQ = kOffK + kKUnits * 2 * kTileBytes;
    static constexpr int kOffL = kOffQ + kQStages * kTileBytes;
    static constexpr int kOffBar = kOffL + kLStages * kLBytes;
    static constexpr int kKFull = 0, kKEmpty = kKFull + 2 * kKUnits;  // full: 2 unit + tile
    static constexpr int kQFull = kKEmpty + kKUnits, kQEmpty = kQFull + kQStages;
    static constexpr int kLFull = kQEmpty + kQStages, kLEmpty = kLFull + kLStages;
    static constexpr int kSFull = kLEmpty + kLStages, kSEmpty = kSFull + 2;  // + buffer
    static constexpr int kPartFull = kSEmpty + 2, kPartEmpty = kPartFull + 1;
    static constexpr int kTeardown = kPartEmpty + 1, kNumBars = kTeardown + 1;
    static constexpr int kOffMisc = (kOffBar + 8 * kNumBars + 15) & ~15;
    static constexpr int kOffSteps = kOffMisc + 16;  // int [kKUnits]: steps of the unit there, 0: no more units
    static constexpr int kOffRun = kOffMisc + 32;
    static constexpr int kOffPart = (kOffRun + static_cast<int>(sizeof(Run)) + 15) & ~15;  // [2][128] sums
    static constexpr int kSmemBytes = kOffPart + 1024;
    static_assert(kSmemBytes <= 227 * 1024 && kPlanBytes <= kOffQ, "shared memory budget");
    static_assert(kKUnits <= 4 && kLStages >= 2);
};

// Tokens [t0, t1) of a chunk that see a key of [k0, k0 + kUnitKeys).
struct Tokens {
    int t0, t1;
    __device__ __forceinline__ Tokens(const PagedParams &p, const Seq &s, int k0) {
        const int pos0 = s.L - s.Lq;
        t0 = max(k0 - pos0, 0);
        t1 = s.Lq;
        if (p.window > 0 && k0 >= p.sinks) t1 = min(t1, max(k0 + kUnitKeys - 1 + p.window - pos0, 0));
    }
    __device__ __forceinline__ int tiles(const PagedParams &p) const {
        return t1 > t0 ? (t1 - t0 + p.tile_tokens - 1) / p.tile_tokens : 0;
    }
};

struct Units {
    const PagedParams &p;
    __device__ __forceinline__ int count(const Seq &s) const { return s.Lq > 0 ? (s.L + kUnitKeys - 1) / kUnitKeys : 0; }
    __device__ __forceinline__ int cost(const Seq &s, int i) const {
        const int n = Tokens(p, s, i * kUnitKeys).tiles(p);
        return n > 0 ? n + kStart : 0;
    }
    // units that all of the chunk sees: from 0 on those that start ahead of it (with a window: and hold sinks)
    __device__ __forceinline__ int2 flat(const Seq &s, int n) const {
        const int pos0 = s.L - s.Lq;
        int to = pos0 >= 0 ? min(n, pos0 / kUnitKeys + 1) : 0;
        if (p.window > 0) to = min(to, (p.sinks + kUnitKeys - 1) / kUnitKeys);
        return make_int2(0, to);
    }
};

// The units that start in a CTA's run; the warps that load walk them, each for itself.
struct Unit {
    int b, hk, k0, steps, t0, t1;
    Seq s;
};

// What the warps that add up need to know of a step: tokens [., . + n) of the
// chunk, the first at position `first`; 0: no more steps.
struct __align__(16) Step {
    int n, first;
    int j, steps;    // the step in its unit, the unit's
    int k0, L, row;  // the unit's first key, the sequence's keys, its row of the weights
    int pad;
};

struct Walk {
    const PagedParams &p;
    long long rem;
    int b, hk, unit, off, n;
    Seq s;

    __device__ __forceinline__ Walk(const PagedParams &p_, const volatile Run *r) : p(p_) {
        rem = r->len;
        b = r->b;
        hk = r->hk;
        unit = r->unit;
        off = r->off;
        n = 0;
        s.q0 = r->s.q0;
        s.Lq = r->s.Lq;
        s.L = r->s.L;
        if (rem > 0) n = Units{p}.count(s);
    }
    __device__ __forceinline__ bool next(Unit &o) {
        while (rem > 0) {
            if (unit >= n) {
                unit = 0;
                if (n == 0 || ++hk == p.Hkv) {
                    hk = 0;
                    if (++b >= p.B) return false;
                    s = load_seq(p, b);
                    n = Units{p}.count(s);
                    continue;
                }
            }
            const Tokens t(p, s, unit * kUnitKeys);
            const int tiles = t.tiles(p), cost = tiles > 0 ? tiles + kStart : 0;
            const bool starts = off == 0 && tiles > 0;
            o = Unit{b, hk, unit * kUnitKeys, tiles, t.t0, t.t1, s};
            rem -= cost - off;
            off = 0;
            ++unit;
            if (starts) return true;
        }
        return false;
    }
};

// Key tile T of each unit, and (T = 1) the query tiles of its steps. One warp for
// both key tiles: 45.4 us for the first of the cases above in place of 42.0.
template <int D, int T>
__device__ void producer(const CUtensorMap *tq, const CUtensorMap *tk, const WeightsParams &p, uint32_t sbase,
                         volatile int *steps, const volatile Run *run, volatile int *abort_flag) {
    using S = Shape<D>;
    auto bar = [&](int i) { return sbase + S::kOffBar + 8u * static_cast<uint32_t>(i); };
    const bool leader = ptx::elect_one();
    const uint32_t bytes = static_cast<uint32_t>(p.tile_tokens * p.group * 128 * S::kColBlocks);
    const Pages pages(p);
    uint32_t units = 0, it = 0;  // loaded: key tiles, query tiles
    bool ok = true;
    Walk walk(p, run);
    Unit u{};
    for (;; ++units) {
        // the next unit's pages are on their way while its place is waited for
        const bool more = walk.next(u);
        if (T == 0 && !more) break;
        const Dead dead(p, u.s);
        const Head at{u.b, u.hk, u.s.L};
        const int k0 = u.k0 + T * kBlockN, page = more ? pages.look_up(p, at, dead, k0) : -1;
        const uint32_t stage = units % S::kKUnits;
        if (units >= S::kKUnits &&
            !(ok = ptx::warp_all(ptx::bar_wait(bar(S::kKEmpty + stage), ((units / S::kKUnits) - 1) & 1, abort_flag,
                                 p.timeout_ns))))
            break;
        const uint32_t dst = sbase + S::kOffK + (2 * stage + T) * S::kTileBytes, full = bar(S::kKFull + 2 * stage + T);
        if (T == 1 && leader) steps[stage] = more ? u.steps : 0;
        if (!more || p.log2_bs < 3) {
            if (more) copy_small_pages<D>(p, at, dead, k0, p.k, dst);
            if (leader) ptx::bar_arrive(full);
        } else {
            if (leader) ptx::bar_arrive_expect_tx(full, S::kTileBytes);
            __syncwarp();
            pages.load<D>(p, at, dead, k0, page, tk, dst, full);
            __syncwarp();
        }
        if (!more) {
            ++units;
            break;
        }
        if (T == 1) {
            for (int j = 0; j < u.steps; ++j, ++it) {
                const uint32_t qs = it % S::kQStages;
                if (it >= S::kQStages &&
                    !(ok = ptx::warp_all(ptx::bar_wait(bar(S::kQEmpty + qs), ((it / S::kQStages) - 1) & 1, abort_flag,
                                         p.timeout_ns))))
                    break;
                if (leader && !withheld(p.withhold, it)) {
                    ptx::bar_arrive_expect_tx(bar(S::kQFull + qs), bytes);
#pragma unroll
                    for (int c = 0; c < S::kColBlocks; ++c)
                        ptx::tma_load_4d(sbase + S::kOffQ + qs * S::kTileBytes + c * S::kBlockBytes, tq,
                                         bar(S::kQFull + qs), c * 64, 0, u.hk, u.s.q0 + u.t0 + j * p.tile_tokens);
                }
            }
            if (!ok) {
                ++units;
                break;
            }
        }
    }
    // never leave with copies in flight (bounded, even after an abort)
    for (uint32_t s = 0; s < S::kKUnits && s < units; ++s) {
        const uint32_t last = (units - 1) - ((units - 1 - s) % S::kKUnits);
        ptx::bar_wait(bar(S::kKFull + 2 * s + T), (last / S::kKUnits) & 1, nullptr, p.timeout_ns);
    }
    for (uint32_t s = 0; T == 1 && s < S::kQStages && s < it; ++s) {
        const uint32_t last = (it - 1) - ((it - 1 - s) % S::kQStages);
        ptx::bar_wait(bar(S::kQFull + s), (last / S::kQStages) & 1, nullptr, p.timeout_ns);
    }
}

// Of each step its Step and -lse log2 e of its columns; -inf for columns that are no
// query, and for queries that see nothing. Then a Step without tokens for each
// warpgroup.
template <int D>
__device__ void producer_lse(const WeightsParams &p, uint32_t sbase, uint8_t *ring, const volatile Run *run,
                             volatile int *abort_flag) {
    using S = Shape<D>;
    auto bar = [&](int i) { return sbase + S::kOffBar + 8u * static_cast<uint32_t>(i); };
    const int lane = threadIdx.x % 32;
    int token[4], head[4];  // of columns lane, lane + 32, ...
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        token[i] = (lane + 32 * i) / p.group;
        head[i] = lane + 32 * i - token[i] * p.group;
    }
    uint32_t it = 0;
    Walk walk(p, run);
    Unit u{};
    int j = 0, end = 0;
    while (end < 2) {
        if (j >= u.steps && end == 0) {
            j = 0;
            if (!walk.next(u)) end = 1;
        } else if (end == 1) {
            end = 2;
        }
        const int t0 = u.t0 + j * p.tile_tokens, n = end > 0 ? 0 : min(p.tile_tokens, u.t1 - t0);
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = CUDART_INF_F;
            if (token[i] < n)
                x[i] = __ldcg(p.lse + static_cast<long long>(u.hk * p.group + head[i]) * p.lse_head +
                              static_cast<long long>(u.s.q0 + t0 + token[i]) * p.lse_token);
        }
        const uint32_t stage = it % S::kLStages;
        if (it >= S::kLStages &&
            !ptx::warp_all(ptx::bar_wait(bar(S::kLEmpty + stage), ((it / S::kLStages) - 1) & 1, abort_flag,
                                         p.timeout_ns)))
            break;
        uint8_t *to = ring + stage * S::kLBytes;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            reinterpret_cast<float *>(to)[lane + 32 * i] =
                x[i] == -CUDART_INF_F ? -CUDART_INF_F : x[i] * -1.4426950408889634f;
        if (lane == 0)
            *reinterpret_cast<Step *>(to + 512) =
                Step{n, u.s.L - u.s.Lq + t0, j, u.steps, u.k0, u.s.L, u.b * p.Hkv + u.hk, 0};
        __syncwarp();
        if (lane == 0) ptx::bar_arrive(bar(S::kLFull + stage));
        ++it;
        ++j;
    }
}

template <int D, bool BF16>
__device__ void mma(const WeightsParams &p, uint32_t sbase, uint32_t tmem, const volatile int *steps,
                    volatile int *abort_flag) {
    using S = Shape<D>;
    auto bar = [&](int i) { return sbase + S::kOffBar + 8u * static_cast<uint32_t>(i); };
    const uint32_t idesc = ptx::idesc_f16(BF16, kBlockN, 32 * p.chunks, false);
    const bool leader = ptx::elect_one();
    const uint64_t dq0 = ptx::smem_desc_sw128(sbase + S::kOffQ, 16, 1024);
    const uint64_t dk0 = ptx::smem_desc_sw128(sbase + S::kOffK, 16, 1024);
    constexpr uint64_t kTile16 = S::kTileBytes >> 4, kBlock16 = S::kBlockBytes >> 4;
    uint32_t it = 0;
    bool ok = true;
    for (uint32_t units = 0; ok; ++units) {
        const uint32_t ks = units % S::kKUnits;
        auto wait_k = [&](int t) {
            return ptx::warp_all(ptx::bar_wait(bar(S::kKFull + 2 * ks + t), (units / S::kKUnits) & 1, abort_flag,
                                               p.timeout_ns));
        };
        if (!(ok = wait_k(1))) break;
        const int n = steps[ks];
        if (n == 0 || !(ok = wait_k(0))) break;
        for (int j = 0; j < n; ++j, ++it) {
            const uint32_t qs = it % S::kQStages, buf = it % 2;
            if (!(ok = ptx::warp_all(ptx::bar_wait(bar(S::kQFull + qs), (it / S::kQStages) & 1, abort_flag, p.timeout_ns))))
                break;
            if (it >= 2 &&
                !(ok = ptx::warp_all(ptx::bar_wait(bar(S::kSEmpty + buf), (it / 2 - 1) & 1, abort_flag, p.timeout_ns))))
                break;
            ptx::tc_fence_after();
            if (leader) {
#pragma unroll 1
                for (int t = 0; t < 2; ++t) {
                    const uint64_t kd = dk0 + (2 * ks + t) * kTile16, qd = dq0 + qs * kTile16;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t off = (kk / 4) * kBlock16 + (kk % 4) * 2;
                        ptx::mma_ss(tmem + 128 * (2 * t + buf), kd + off, qd + off, idesc, kk > 0);
                    }
                }
                ptx::mma_commit(bar(S::kSFull + buf));
                ptx::mma_commit(bar(S::kQEmpty + qs));
                if (j + 1 == n) ptx::mma_commit(bar(S::kKEmpty + ks));
            }
        }
    }
    if (leader) ptx::mma_commit(bar(S::kTeardown));
    __syncwarp();
    ptx::bar_wait(bar(S::kTeardown), 0, nullptr, p.timeout_ns);
}

__device__ __forceinline__ void load_pairs(uint32_t at, uint64_t (&x)[2]) {
    asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(x[0]), "=l"(x[1]) : "r"(at));
}

// Zeros for the keys that no unit writes: those behind a sequence, and its units
// that no query sees. Threads [first, kThreads) of all CTAs share the rows.
__device__ __forceinline__ void clear_rest(const WeightsParams &p, int first) {
    const int threads = kThreads - first, width = p.max_blocks << p.log2_bs;
    const long long rows = static_cast<long long>(p.B) * p.Hkv;
    for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
        const Seq s = load_seq(p, static_cast<int>(row / p.Hkv));
        float *w = p.weights + static_cast<size_t>(row) * width;
        const int seen = s.Lq > 0 ? s.L : 0;
        for (int k = seen + threadIdx.x - first; k < width; k += threads) w[k] = 0.f;
        if (p.window == 0 && s.L >= s.Lq) continue;  // a query sees every key
        for (int k = threadIdx.x - first; k < seen; k += threads)
            if (Tokens(p, s, k / kUnitKeys * kUnitKeys).tiles(p) == 0) w[k] = 0.f;
    }
}

// Sums of both key tiles' rows over every second step: a thread has a key of each.
// The two warpgroups are a step apart, so one waits for its scores while the other
// keeps the exponentials going. Who takes a unit's first step writes its sums.
template <int D>
__device__ void sums(const WeightsParams &p, uint32_t sbase, uint32_t tmem, float *part, const uint8_t *ring, uint32_t mine,
                     int wq, int lane, volatile int *abort_flag) {
    using S = Shape<D>;
    auto bar = [&](int i) { return sbase + S::kOffBar + 8u * static_cast<uint32_t>(i); };
    const uint32_t tS = tmem + (static_cast<uint32_t>(wq * 32) << 16) + 128 * mine;
    const int row = wq * 32 + lane;
    const uint64_t scale2 = ptx::pk2(p.scale_log2, p.scale_log2);
    uint32_t shared = 0;  // units whose steps both warpgroups took
    float before[2], sum[2][4];  // of column c: c % 4
    for (uint32_t it = mine;; it += 2) {
        const uint32_t ls = it % S::kLStages;
        bool ok = ptx::bar_wait(bar(S::kLFull + ls), (it / S::kLStages) & 1, abort_flag, p.timeout_ns);
        if (!__all_sync(kFull, ok)) break;
        const Step u = *reinterpret_cast<const Step *>(ring + ls * S::kLBytes + 512);
        if (u.n == 0) break;
        const bool writes = u.j % 2 == 0;
        const int key = u.k0 + row;  // and key + kBlockN
        float *w = p.weights + static_cast<size_t>(u.row) * (static_cast<size_t>(p.max_blocks) << p.log2_bs);
        if (u.j < 2) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                before[t] = 0.f;
                if (p.add && writes && key + t * kBlockN < u.L) before[t] = w[key + t * kBlockN];  // (ahead of its use)
#pragma unroll
                for (int c = 0; c < 4; ++c) sum[t][c] = 0.f;
            }
        }
        ok = ptx::bar_wait(bar(S::kSFull + mine), (it / 2) & 1, abort_flag, p.timeout_ns);
        if (!__all_sync(kFull, ok)) break;
        ptx::tc_fence_after();
        const uint32_t nl_at = sbase + S::kOffL + ls * S::kLBytes;
        // the weights of columns with scores a and b, and -lse in nl
        auto exps = [&](uint32_t a, uint32_t b, uint64_t nl, float &e0, float &e1) {
            float x0, x1;
            ptx::upk2(ptx::ffma2(ptx::pk2(__uint_as_float(a), __uint_as_float(b)), scale2, nl), x0, x1);
            e0 = ptx::ex2(x0);
            e1 = ptx::ex2(x1);
        };
        // Some columns do not count for some keys: queries ahead of a key or too far
        // behind it, columns that are no query of the chunk but hold one's row (a
        // chunk's last step), or nobody's (an odd number of 32s).
        const bool masked = u.n < p.tile_tokens || u.k0 + kUnitKeys - 1 > u.first || p.chunks % 2 != 0 ||
                            (p.window > 0 && u.k0 + kUnitKeys > p.sinks && u.k0 <= u.first + u.n - 1 - p.window);
        if (masked) {
            int c0[2], c1[2];  // the columns that see the two keys
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int k = key + t * kBlockN;
                c0[t] = min(max(k - u.first, 0), 128) * p.group;
                c1[t] = u.n;
                if (p.window > 0 && k >= p.sinks) c1[t] = min(c1[t], max(k + p.window - u.first, 0));
                c1[t] *= p.group;
            }
#pragma unroll 1
            for (int b = 0; b < u.n * p.group; b += 16) {
                uint32_t x[2][16];
#pragma unroll
                for (int t = 0; t < 2; ++t) ptx::tmem_ld16(tS + 256 * t + b, x[t]);
                ptx::tmem_ld_wait();
                ptx::reg_fence(x[0]);
                ptx::reg_fence(x[1]);
                uint32_t seen[2];  // its bits of these columns
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    auto below = [&](int c) { return (1u << min(max(c - b, 0), 16)) - 1; };
                    seen[t] = below(c1[t]) & ~below(c0[t]);
                }
#pragma unroll
                for (int c = 0; c < 16; c += 4) {
                    uint64_t nl[2];
                    load_pairs(nl_at + 4 * (b + c), nl);
#pragma unroll
                    for (int h = 0; h < 4; h += 2)
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            float e0, e1;
                            exps(x[t][c + h], x[t][c + h + 1], nl[h / 2], e0, e1);
                            sum[t][h] += seen[t] >> (c + h) & 1 ? e0 : 0.f;
                            sum[t][h + 1] += seen[t] >> (c + h) & 2 ? e1 : 0.f;
                        }
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::bar_arrive(bar(S::kSEmpty + mine));
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (c >= p.chunks) break;
                uint32_t x[2][32];
#pragma unroll
                for (int t = 0; t < 2; ++t) ptx::tmem_ld32(tS + 256 * t + 32 * c, x[t]);
                ptx::tmem_ld_wait();
                ptx::reg_fence(x[0]);
                ptx::reg_fence(x[1]);
                if (c + 1 == p.chunks) {
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::bar_arrive(bar(S::kSEmpty + mine));
                }
#pragma unroll
                for (int d = 0; d < 32; d += 4) {
                    uint64_t nl[2];
                    load_pairs(nl_at + 128 * c + 4 * d, nl);
#pragma unroll
                    for (int h = 0; h < 4; h += 2)
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            float e0, e1;
                            exps(x[t][d + h], x[t][d + h + 1], nl[h / 2], e0, e1);
                            sum[t][h] += e0;
                            sum[t][h + 1] += e1;
                        }
                }
            }
        }
        __syncwarp();
        if (lane == 0) ptx::bar_arrive(bar(S::kLEmpty + ls));
        if (u.j + 2 < u.steps) continue;
        // this warpgroup's last step of the unit
        float total[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) total[t] = (sum[t][0] + sum[t][1]) + (sum[t][2] + sum[t][3]);
        if (u.steps > 1) {
            // The other's sums go through shared memory to the one that writes. Both wait
            // for the unit before to be through: neither barrier is then more than a
            // phase away.
            ok = shared == 0 || ptx::bar_wait(bar(S::kPartEmpty), (shared - 1) & 1, abort_flag, p.timeout_ns);
            ok = ok && (!writes || ptx::bar_wait(bar(S::kPartFull), shared & 1, abort_flag, p.timeout_ns));
            if (!__all_sync(kFull, ok)) break;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (writes) total[t] += part[t * kBlockN + row];
                else part[t * kBlockN + row] = total[t];
            }
            __syncwarp();
            if (lane == 0) ptx::bar_arrive(bar(writes ? S::kPartEmpty : S::kPartFull));
            ++shared;
        }
        if (writes) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (key + t * kBlockN < u.L) w[key + t * kBlockN] = before[t] + total[t];
        }
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    fa_kv_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const WeightsParams p) {
    using S = Shape<D>;
    extern __shared__ __align__(1024) uint8_t smem[];  // (there is no room to align it)
    const uint32_t sbase = ptx::smem_addr(smem);
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    if ((sbase & 1023) != 0) {
        if (threadIdx.x == 0) atomicExch(p.err, kDeviceErrLaunch);
        return;
    }
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + S::kOffMisc + 4);
    Run *run = reinterpret_cast<Run *>(smem + S::kOffRun);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    // the plan's scratch lies where the keys go
    plan(p, Units{p}, run, smem);
    if (warp == 1) {
        if (lane == 0) {
            for (int i = 0; i < S::kNumBars; ++i) {
                const bool s_empty = i >= S::kSEmpty && i < S::kPartFull, l_empty = i >= S::kLEmpty && i < S::kSFull;
                const bool sums = i >= S::kPartFull && i < S::kTeardown;
                // one arrival per warp
                ptx::bar_init(sbase + S::kOffBar + 8u * i, s_empty || l_empty || sums ? 4u : 1u);
            }
            *abort_flag = 0;
            ptx::bar_init_fence();
        }
        __syncwarp();
        ptx::tmem_alloc(ptx::smem_addr(tmem_slot), 512);
        ptx::tmem_relinquish();
    } else if (warp == 2 && lane == 0) {
        ptx::prefetch_tmap(&tm_q);
        ptx::prefetch_tmap(&tm_k);
    } else if (warp >= 4 && warp < 4 + S::kQStages) {
        // rows that no box reaches are zeros: their scores are finite, their weights 0
        ptx::zero_rows(sbase + S::kOffQ + (warp - 4) * S::kTileBytes, S::kColBlocks, kBlockM, p.tile_tokens * p.group,
                       kBlockM);
    }
    ptx::fence_proxy_async_smem();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    volatile int *steps = reinterpret_cast<volatile int *>(smem + S::kOffSteps);
    if (warp == 0) producer<D, 0>(&tm_q, &tm_k, p, sbase, steps, run, abort_flag);
    else if (warp == 1) mma<D, BF16>(p, sbase, tmem, steps, abort_flag);
    else if (warp == 2) producer_lse<D>(p, sbase, smem + S::kOffL, run, abort_flag);
    else if (warp == 3) producer<D, 1>(&tm_q, &tm_k, p, sbase, steps, run, abort_flag);
    else {
        if (!p.add && run->per > 0) clear_rest(p, 128);  // (while the first keys are on their way)
        sums<D>(p, sbase, tmem, reinterpret_cast<float *>(smem + S::kOffPart), smem + S::kOffL, (warp - 4) / 4, warp % 4,
                lane, abort_flag);
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && *abort_flag) atomicExch(p.err, kDeviceErrTimeout);
}

template <int D, bool BF16>
static cudaError_t launch_t(const CUtensorMap *maps, const WeightsParams &p, int grid, cudaStream_t st) {
    static std::atomic<unsigned long long> done{0};
    auto kern = fa_kv_weights_kernel<D, BF16>;
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kern), Shape<D>::kSmemBytes, done);
    if (e != cudaSuccess) return e;
    return launch_early(kern, dim3(static_cast<unsigned>(grid)), kThreads, Shape<D>::kSmemBytes, st, true, maps[0],
                        maps[1], p);
}

}  // namespace weights

cudaError_t launch_kv_weights(int D, bool bf16, const CUtensorMap *maps, WeightsParams p, int grid, cudaStream_t st) {
    p.chunks = (p.tile_tokens * p.group + 31) / 32;
    if (D == 64)
        return bf16 ? weights::launch_t<64, true>(maps, p, grid, st) : weights::launch_t<64, false>(maps, p, grid, st);
    return bf16 ? weights::launch_t<128, true>(maps, p, grid, st) : weights::launch_t<128, false>(maps, p, grid, st);
}

}  // namespace fa
