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
// Bound: single tokens by reading the keys (16 sequences of 4100 to 8192 keys, 8 key
// heads, D = 128: 47 us, 4.4 TB/s, of which 8 us are the launch and the way to the first
// keys). Long chunks by the exponentials: 512 tokens of four sequences of 8704 to 16896
// keys, 32 heads on 8, take 210 us, 1190 TFLOP/s, 53 % of the rate of ex2; without the
// products 204, products and loads alone 169 (both operands come from shared memory).
// Measured beside this: both warpgroups on every step, half of the columns each, 229;
// a step's scores loaded while the step before is added up, 265 to 317; sums two at a
// time 248; four warpgroups 225.
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
    static constexpr int kLStages = 3;
    static constexpr int kOffK = 0;
    static constexpr int kOffQ = kOffK + kKUnits * 2 * kTileBytes;
    static constexpr int kOffL = kOffQ + kQStages * kTileBytes;
    static constexpr int kOffBar = kOffL + kLStages * 512;
    static constexpr int kKFull = 0, kKEmpty = kKFull + 2 * kKUnits;  // full: 2 unit + tile
    static constexpr int kQFull = kKEmpty + kKUnits, kQEmpty = kQFull + kQStages;
    static constexpr int kLFull = kQEmpty + kQStages, kLEmpty = kLFull + kLStages;
    static constexpr int kSFull = kLEmpty + kLStages, kSEmpty = kSFull + 2;  // + buffer
    static constexpr int kPartFull = kSEmpty + 2, kPartEmpty = kPartFull + 1;
    static constexpr int kTeardown = kPartEmpty + 1, kNumBars = kTeardown + 1;
    static constexpr int kOffMisc = (kOffBar + 8 * kNumBars + 15) & ~15;
    static constexpr int kOffRun = kOffMisc + 16;
    static constexpr int kOffPart = (kOffRun + static_cast<int>(sizeof(Run)) + 15) & ~15;  // [2][128] sums
    static constexpr int kSmemBytes = kOffPart + 1024;
    static_assert(kSmemBytes <= 227 * 1024 && kPlanBytes <= kOffQ, "shared memory budget");
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

// The units that start in a CTA's run; every role walks them for itself.
struct Unit {
    int b, hk, k0, steps, t0, t1;
    Seq s;
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
// both key tiles issues 16-key pages' boxes (32 a unit) no faster than 5.4 TB/s; two
// get 6.4.
template <int D, int T>
__device__ void producer(const CUtensorMap *tq, const CUtensorMap *tk, const WeightsParams &p, uint32_t sbase,
                         const volatile Run *run, volatile int *abort_flag) {
    using S = Shape<D>;
    auto bar = [&](int i) { return sbase + S::kOffBar + 8u * static_cast<uint32_t>(i); };
    const bool leader = ptx::elect_one();
    const uint32_t bytes = static_cast<uint32_t>(p.tile_tokens * p.group * 128 * S::kColBlocks);
    const Pages pages(p);
    uint32_t units = 0, it = 0;  // loaded: key tiles, query tiles
    bool ok = true;
    Walk walk(p, run);
    // a unit's pages are looked up while the one before it is waited for and loaded
    Unit u, after;
    int page = -1, page_after = -1;
    auto look_up = [&](const Unit &x) {
        return pages.look_up(p, Head{x.b, x.hk, x.s.L}, Dead(p, x.s), x.k0 + T * kBlockN);
    };
    bool more = walk.next(u);
    if (more) page = look_up(u);
    for (; more; ++units) {
        bool next = false;
        auto look_ahead = [&] {
            next = walk.next(after);
            if (next) page_after = look_up(after);
        };
        if (units > 0) look_ahead();  // (the first is not kept waiting)
        const Dead dead(p, u.s);
        const Head at{u.b, u.hk, u.s.L};
        const uint32_t stage = units % S::kKUnits;
        if (units >= S::kKUnits &&
            !(ok = ptx::warp_all(ptx::bar_wait(bar(S::kKEmpty + stage), ((units / S::kKUnits) - 1) & 1, abort_flag,
                                 p.timeout_ns))))
            break;
        const uint32_t dst = sbase + S::kOffK + (2 * stage + T) * S::kTileBytes, full = bar(S::kKFull + 2 * stage + T);
        if (p.log2_bs < 3) {
            copy_small_pages<D>(p, at, dead, u.k0 + T * kBlockN, p.k, dst);
            if (leader) ptx::bar_arrive(full);
        } else {
            if (leader) ptx::bar_arrive_expect_tx(full, S::kTileBytes);
            __syncwarp();
            pages.load<D>(p, at, dead, u.k0 + T * kBlockN, page, tk, dst, full);
            __syncwarp();
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
        }
        if (units == 0) look_ahead();
        if (!ok) {
            ++units;
            break;
        }
        more = next;
        u = after;
        page = page_after;
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

// -lse log2 e of each column of each step; -inf for columns that are no query,
// and for queries that see nothing.
template <int D>
__device__ void producer_lse(const WeightsParams &p, uint32_t sbase, float *ring, const volatile Run *run,
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
    bool ok = true;
    Walk walk(p, run);
    Unit u{};
    int j = 0;
    // values of the step at (u, j), which moves on; a step's are loaded while the
    // ring's place for the one before it is waited for
    auto load = [&](float (&x)[4]) {
        const int t0 = u.t0 + j * p.tile_tokens, n = min(p.tile_tokens, u.t1 - t0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = CUDART_INF_F;
            if (token[i] < n)
                x[i] = __ldcg(p.lse + static_cast<long long>(u.hk * p.group + head[i]) * p.lse_head +
                             static_cast<long long>(u.s.q0 + t0 + token[i]) * p.lse_token);
        }
        if (++j < u.steps) return true;
        j = 0;
        return walk.next(u);
    };
    float x[4], after[4];
    bool more = walk.next(u), next = false;
    if (more) next = load(x);
    for (; more; ++it) {
        more = next;
        if (more) next = load(after);
        const uint32_t stage = it % S::kLStages;
        if (it >= S::kLStages &&
            !(ok = ptx::warp_all(ptx::bar_wait(bar(S::kLEmpty + stage), ((it / S::kLStages) - 1) & 1, abort_flag,
                                 p.timeout_ns))))
            break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ring[stage * 128 + lane + 32 * i] = x[i] == -CUDART_INF_F ? -CUDART_INF_F : x[i] * -1.4426950408889634f;
            x[i] = after[i];
        }
        __syncwarp();
        if (lane == 0) ptx::bar_arrive(bar(S::kLFull + stage));
    }
}

template <int D, bool BF16>
__device__ void mma(const WeightsParams &p, uint32_t sbase, uint32_t tmem, const volatile Run *run,
                    volatile int *abort_flag) {
    using S = Shape<D>;
    auto bar = [&](int i) { return sbase + S::kOffBar + 8u * static_cast<uint32_t>(i); };
    const uint32_t idesc = ptx::idesc_f16(BF16, kBlockN, 32 * p.chunks, false);
    const bool leader = ptx::elect_one();
    const uint64_t dq0 = ptx::smem_desc_sw128(sbase + S::kOffQ, 16, 1024);
    const uint64_t dk0 = ptx::smem_desc_sw128(sbase + S::kOffK, 16, 1024);
    constexpr uint64_t kTile16 = S::kTileBytes >> 4, kBlock16 = S::kBlockBytes >> 4;
    uint32_t units = 0, it = 0;
    bool ok = true;
    Walk walk(p, run);
    Unit u;
    for (; ok && walk.next(u); ++units) {
        const uint32_t ks = units % S::kKUnits;
#pragma unroll
        for (int t = 0; t < 2; ++t)
            ok = ok && ptx::warp_all(ptx::bar_wait(bar(S::kKFull + 2 * ks + t), (units / S::kKUnits) & 1, abort_flag,
                                                   p.timeout_ns));
        if (!ok) break;
        for (int j = 0; j < u.steps; ++j, ++it) {
            const uint32_t qs = it % S::kQStages, buf = it % 2;
            if (!(ok = ptx::warp_all(ptx::bar_wait(bar(S::kQFull + qs), (it / S::kQStages) & 1, abort_flag, p.timeout_ns))))
                break;
            if (it >= 2 &&
                !(ok = ptx::warp_all(ptx::bar_wait(bar(S::kSEmpty + buf), (it / 2 - 1) & 1, abort_flag, p.timeout_ns))))
                break;
            ptx::tc_fence_after();
            if (leader) {
#pragma unroll
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
                if (j + 1 == u.steps) ptx::mma_commit(bar(S::kKEmpty + ks));
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
// keeps the exponentials going.
template <int D>
__device__ void sums(const WeightsParams &p, uint32_t sbase, uint32_t tmem, float *part, uint32_t mine, int wq,
                     int lane, const volatile Run *run, volatile int *abort_flag) {
    using S = Shape<D>;
    auto bar = [&](int i) { return sbase + S::kOffBar + 8u * static_cast<uint32_t>(i); };
    const uint32_t tS = tmem + (static_cast<uint32_t>(wq * 32) << 16) + 128 * mine;
    const int row = wq * 32 + lane;
    const uint64_t scale2 = ptx::pk2(p.scale_log2, p.scale_log2);
    uint32_t it = 0, shared = 0;  // steps; units whose steps both warpgroups took
    bool ok = true;
    Walk walk(p, run);
    Unit u;
    while (ok && walk.next(u)) {
        const int pos0 = u.s.L - u.s.Lq, key = u.k0 + row;  // and key + kBlockN
        float *w = p.weights + (static_cast<size_t>(u.b) * p.Hkv + u.hk) * (static_cast<size_t>(p.max_blocks) << p.log2_bs);
        // who writes the unit's sums: the one that takes its first step
        const bool writes = it % 2 == mine;
        float before[2] = {0.f, 0.f};
        if (p.add && writes) {  // (ahead of their use)
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (key + t * kBlockN < u.s.L) before[t] = w[key + t * kBlockN];
        }
        float sum[2][4] = {};  // of column c: c % 4
        for (int j = writes ? 0 : 1; j < u.steps; j += 2) {
            const uint32_t i = it + j, ls = i % S::kLStages;
            ok = ptx::bar_wait(bar(S::kLFull + ls), (i / S::kLStages) & 1, abort_flag, p.timeout_ns) &&
                 ptx::bar_wait(bar(S::kSFull + mine), (i / 2) & 1, abort_flag, p.timeout_ns);
            if (!__all_sync(kFull, ok)) { ok = false; break; }
            ptx::tc_fence_after();
            const int t0 = u.t0 + j * p.tile_tokens, n = min(p.tile_tokens, u.t1 - t0), first = pos0 + t0;
            const uint32_t nl_at = sbase + S::kOffL + ls * 512;
            // the weights of columns c and c + 1 of the 32 in x
            auto exps = [&](const uint32_t (&x)[32], int c, uint64_t nl, float &e0, float &e1) {
                float x0, x1;
                ptx::upk2(ptx::ffma2(ptx::pk2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), scale2, nl), x0, x1);
                e0 = ptx::ex2(x0);
                e1 = ptx::ex2(x1);
            };
            // Some columns do not count for some keys: queries ahead of a key or too far
            // behind it, columns that are no query of the chunk but hold one's row (a
            // chunk's last step), or nobody's (an odd number of 32s).
            const bool masked = n < p.tile_tokens || u.k0 + kUnitKeys - 1 > first || p.chunks % 2 != 0 ||
                                (p.window > 0 && u.k0 + kUnitKeys > p.sinks && u.k0 <= first + n - 1 - p.window);
            if (masked) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int k = key + t * kBlockN;  // seen by the columns [c0, c1)
                    const int c0 = min(max(k - first, 0), 128) * p.group;
                    int c1 = n;
                    if (p.window > 0 && k >= p.sinks) c1 = min(c1, max(k + p.window - first, 0));
                    c1 *= p.group;
#pragma unroll 1
                    for (int b = 0; b < p.chunks; ++b) {
                        auto below = [&](int c) { return static_cast<uint32_t>((1ull << min(max(c - 32 * b, 0), 32)) - 1); };
                        const uint32_t seen = below(c1) & ~below(c0);
                        uint32_t x[32];
                        ptx::tmem_ld32(tS + 256 * t + 32 * b, x);
                        ptx::tmem_ld_wait();
                        ptx::reg_fence(x);
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            uint64_t nl[2];
                            load_pairs(nl_at + 128 * b + 4 * c, nl);
#pragma unroll
                            for (int h = 0; h < 4; h += 2) {
                                float e0, e1;
                                exps(x, c + h, nl[h / 2], e0, e1);
                                sum[t][h] += seen >> (c + h) & 1 ? e0 : 0.f;
                                sum[t][h + 1] += seen >> (c + h) & 2 ? e1 : 0.f;
                            }
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
                                exps(x[t], d + h, nl[h / 2], e0, e1);
                                sum[t][h] += e0;
                                sum[t][h + 1] += e1;
                            }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) ptx::bar_arrive(bar(S::kLEmpty + ls));
        }
        if (!ok) break;
        it += u.steps;
        float total[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) total[t] = (sum[t][0] + sum[t][1]) + (sum[t][2] + sum[t][3]);
        if (u.steps > 1) {
            // The other's sums go through shared memory to the one that writes. Both wait
            // for the unit before to be through: neither barrier is then more than a
            // phase away.
            ok = shared == 0 || ptx::bar_wait(bar(S::kPartEmpty), (shared - 1) & 1, abort_flag, p.timeout_ns);
            ok = ok && (!writes || ptx::bar_wait(bar(S::kPartFull), shared & 1, abort_flag, p.timeout_ns));
            if (!__all_sync(kFull, ok)) { ok = false; break; }
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
                if (key + t * kBlockN < u.s.L) w[key + t * kBlockN] = before[t] + total[t];
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
        if (threadIdx.x == 0) atomicExch(p.err, kDeviceErrTimeout);
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

    if (warp == 0) producer<D, 0>(&tm_q, &tm_k, p, sbase, run, abort_flag);
    else if (warp == 1) mma<D, BF16>(p, sbase, tmem, run, abort_flag);
    else if (warp == 2) producer_lse<D>(p, sbase, reinterpret_cast<float *>(smem + S::kOffL), run, abort_flag);
    else if (warp == 3) producer<D, 1>(&tm_q, &tm_k, p, sbase, run, abort_flag);
    else {
        if (!p.add && run->per > 0) clear_rest(p, 128);  // (while the first keys are on their way)
        sums<D>(p, sbase, tmem, reinterpret_cast<float *>(smem + S::kOffPart), (warp - 4) / 4, warp % 4, lane, run,
                abort_flag);
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
