// Attention of chunks of new tokens over a paged cache (fa_fwd_paged), tcgen05
// with TMEM accumulators.
//
// Query t of a sequence's chunk is at position L - Lq + t of its L keys and sees
// key j if j <= its position and (that is less than `window` away, or window is
// 0, or j < sinks). The roles, barriers, TMEM columns and the online softmax are
// those of the packed forward (fa_fwd_kernel.cuh); what differs:
//
// Rows. A query tile holds the group's query heads of consecutive tokens (row =
// token * group + head of the group, floor(128 / group) tokens), so that few
// tokens still fill a tile and a key head is read once for all of its query
// heads. One 4-D TMA box brings it.
//
// Pages. A 128-key tile of K or V is brought page by page (a lane looks up and
// loads one page; pages of 128 keys and more: the part of one). Keys that no
// query of the chunk sees are zeros: whole pages of them are not looked up, a
// box outside the tensor stands for them, and V's rows are cleared behind the
// load. Pages of less than 8 rows do not fill a swizzle atom and go through
// 16-byte asynchronous copies.
//
// Work. Lengths are on the device, so the kernel cuts the work itself: units
// (sequence, key head, pair of query tiles), each as long as the key tiles it
// visits and kStart, are laid end to end and cut into equal runs, one per CTA,
// so that one long sequence or many ragged ones keep every SM busy to the end. A
// unit that falls into several runs leaves its parts (m, l, O in fp32) in the
// workspace, and a second launch joins them, in a fixed order.
//
// Rounding. P is rounded to the 16-bit type once, ahead of P V, as in the packed
// forward: o is then off by 2.3e-3 (root mean square, bf16; 2.7e-4 fp16) where 32-bit
// products would leave 1.7e-3 (2.1e-4), o's own rounding. P as two 16-bit numbers, as the
// paged decode of single tokens takes it, would be half as many products again: 551 us ->
// 826 at the tensor core's rate for the long chunk below.
//
// Bound: long chunks by the tensor core under the power limit, 2048 tokens behind 30000
// keys, 32 heads on 8 of D = 128: 631 us, 1650 TFLOP/s, sustained 680 to 717. 16 chunks of 1 to 512 tokens
// behind up to 7680 keys: 294 us, 1260 TFLOP/s (tensor core 65 % active: starts of units,
// rows without tokens, keys ahead of the chunk's queries). Few tokens by reading the
// cache: 5 of 16 sequences of up to 8192 keys 79 us, 5.1 TB/s, of which 20 are the launch,
// the plan, the first loads and the join (at 32000 keys 314 us, 6.7 TB/s).
// Measured beside this: units in groups of sequences, so that neighbours share keys in
// L2, 294 and 640 to 660; the softmax warps' place in the run kept in registers, 920
// (spills) in place of 680; one warpgroup after the other where a unit is one tile, no
// gain; a start that counts as 1, 2 or 4 tiles, slower.
#pragma once

#include "fa_paged.cuh"

namespace fa {
namespace chunk {

using namespace paged;

// What a unit's start (its queries, first keys, and end) costs, in key tiles.
constexpr int kStart = 3;

__device__ __forceinline__ int pairs_of(const ChunkParams &p, const Seq &s) {
    return (s.Lq + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens);
}

// Key tiles of a unit: its steps are tiles [0, ns), which hold sinks, then the
// tiles from lo on; query tile t visits tiles [0, sink[t]) and [wlo[t], hi[t]).
struct Tiles {
    int tok[2], ntok[2];  // first token of each query tile (in the chunk), tokens
    int ns, lo, steps;
    int sink[2], wlo[2], hi[2];
};

__device__ __forceinline__ Tiles tiles_of(const ChunkParams &p, const Seq &s, int pair) {
    Tiles k;
    const int pos0 = s.L - s.Lq;
    const int sink_tiles = p.window > 0 ? p.sinks / kBlockN + (p.sinks % kBlockN != 0) : 0;
    int end = 0;
    k.ns = 0;
    k.lo = INT_MAX;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        k.tok[t] = (2 * pair + t) * p.tile_tokens;
        k.ntok[t] = min(max(s.Lq - k.tok[t], 0), p.tile_tokens);
        const int first = pos0 + k.tok[t], last = first + k.ntok[t] - 1;
        k.hi[t] = k.ntok[t] > 0 && last >= 0 ? last / kBlockN + 1 : 0;
        k.wlo[t] = p.window > 0 ? max(first - p.window + 1, 0) / kBlockN : 0;
        k.sink[t] = min(sink_tiles, k.hi[t]);
        if (k.hi[t] > 0) {
            k.ns = max(k.ns, k.sink[t]);
            k.lo = min(k.lo, k.wlo[t]);
            end = max(end, k.hi[t]);
        }
    }
    k.lo = max(min(k.lo, end), k.ns);
    k.steps = k.ns + max(end - k.lo, 0);
    return k;
}

__device__ __forceinline__ int tile_at(const Tiles &k, int j) { return j < k.ns ? j : j - k.ns + k.lo; }

__device__ __forceinline__ bool visits(const Tiles &k, int t, int j) {
    const int x = tile_at(k, j);
    return x < k.hi[t] && (x < k.sink[t] || x >= k.wlo[t]);
}

// Steps of [s0, s1) that query tile t visits.
__device__ __forceinline__ int visited(const Tiles &k, int t, int s0, int s1) {
    auto both = [&](int a, int b) { return max(min(b, s1) - max(a, s0), 0); };
    const int from = max(k.wlo[t], k.sink[t]);
    return both(0, k.sink[t]) + both(from, min(k.hi[t], k.ns)) +
           both(max(from, k.lo) - k.lo + k.ns, k.hi[t] - k.lo + k.ns);
}

// What the plan lays out: pairs of query tiles.
struct Units {
    const ChunkParams &p;
    __device__ __forceinline__ int count(const Seq &s) const { return pairs_of(p, s); }
    __device__ __forceinline__ int cost(const Seq &s, int i) const { return tiles_of(p, s, i).steps + kStart; }
    __device__ __forceinline__ int2 flat(const Seq &, int) const { return make_int2(0, 0); }
};

// The parts of a CTA's run, in order; every role walks them for itself.
struct Part {
    int b, hk, pair;
    Seq s;
    Tiles k;
    int s0, s1;   // steps
    bool whole;   // the unit's only part
    int slot;     // of the CTA's two in the workspace, else
    int parts;    // first of several parts: their number, else 0
};

// Where a role is in its CTA's run.
struct Walk {
    long long rem, per;
    int b, hk, pair, off, pairs, first;
    Seq s;

    __device__ __forceinline__ void start(const ChunkParams &p, const volatile Run *r) {
        rem = r->len;
        per = r->per;
        b = r->b;
        hk = r->hk;
        pair = r->unit;
        off = r->off;
        first = 1;
        pairs = 0;
        s.q0 = r->s.q0;
        s.Lq = r->s.Lq;
        s.L = r->s.L;
        if (rem > 0) pairs = pairs_of(p, s);
    }
    __device__ __forceinline__ bool next(const ChunkParams &p, Part &o) {
        while (rem > 0) {
            while (pairs == 0) {  // a sequence without queries
                if (++b >= p.B) return false;
                s = load_seq(p, b);
                pairs = pairs_of(p, s);
            }
            o.b = b;
            o.hk = hk;
            o.pair = pair;
            o.s = s;
            o.k = tiles_of(p, s, pair);
            const int n = o.k.steps + kStart;
            const int take = static_cast<int>(min(rem, static_cast<long long>(n - off)));
            o.s0 = max(off - kStart, 0);
            o.s1 = max(off + take - kStart, 0);
            o.whole = o.s0 == 0 && o.s1 == o.k.steps;
            o.slot = first ? 0 : 1;
            const int rest = n - off - take;
            o.parts = o.s0 == 0 && o.s1 > 0 && rest > 0 ? 1 + static_cast<int>((rest + per - 1) / per) : 0;
            const bool some = o.s1 > o.s0 || (o.k.steps == 0 && off == 0);
            rem -= take;
            first = 0;
            off = 0;
            if (++pair == pairs) {
                pair = 0;
                if (++hk == p.Hkv) {
                    hk = 0;
                    pairs = 0;  // the next sequence is loaded when it is reached
                }
            }
            if (some) return true;
        }
        return false;
    }
};

// A softmax warp's place in the run and what its part needs at the end: kept in
// shared memory while the steps need the registers.
struct Kept {
    Walk walk;
    int tok0, ntok, h0, dest;  // packed row of the tile's first token; tokens; first head; slot, or -1: the unit's only part
};

// Shared memory behind the barriers.
struct Shared {
    Run run;
    Kept kept[8];
};

// ------------------------------------------------------------------ roles --

template <int D>
__device__ void producer_qk(const CUtensorMap *tq, const CUtensorMap *tk, const ChunkParams &p, uint32_t sbase,
                            const volatile Run *run, volatile int *abort_flag) {
    using S = FwdShape<D>;
    const uint32_t bars = sbase + S::kOffBar;
    auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
    const bool leader = ptx::elect_one();
    const uint64_t stream_pol = ptx::l2_policy_evict_first();
    const Pages pages(p);
    const uint32_t tile_q = static_cast<uint32_t>(p.tile_tokens * p.group * 128 * S::kColBlocks);
    uint32_t it = 0, wi = 0, nq = 0;  // K tiles issued, parts loaded, Q loads issued
    bool ok = true;
    Walk walk;
    walk.start(p, run);
    Part u;
    while (ok && walk.next(p, u)) {
        if (u.s1 == u.s0) continue;
        const Dead dead(p, u.s);
        const Head at{u.b, u.hk, u.s.L};
        auto load_q = [&]() -> bool {
            if (nq > 0 &&
                !ptx::warp_all(ptx::bar_wait(bar(S::kQEmpty), (nq - 1) & 1, abort_flag, p.timeout_ns)))
                return false;
            uint32_t bytes = 0;
#pragma unroll
            for (int t = 0; t < 2; ++t) bytes += visited(u.k, t, u.s0, u.s1) > 0 ? tile_q : 0;
            if (leader) ptx::bar_arrive_expect_tx(bar(S::kQFull), bytes);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (visited(u.k, t, u.s0, u.s1) == 0 || !leader) continue;
#pragma unroll
                for (int c = 0; c < S::kColBlocks; ++c)
                    ptx::tma_load_4d_hint(sbase + S::kOffQ + t * S::kTileBytes + c * S::kBlockBytes, tq, bar(S::kQFull),
                                          c * 64, 0, u.hk, u.s.q0 + u.k.tok[t], stream_pol);
            }
            ++nq;
            return true;
        };
        if (wi == 0 && !(ok = load_q())) break;
        int page = pages.look_up(p, at, dead, tile_at(u.k, u.s0) * kBlockN);
        for (int j = u.s0; j < u.s1; ++j, ++it) {
            // the first products need Q and the first K tile only (see the packed forward)
            if (wi == 0 && j == u.s0 + 1 &&
                !(ok = ptx::warp_all(ptx::bar_wait(bar(S::kQFull), 0, abort_flag, p.timeout_ns))))
                break;
            const uint32_t stage = it % S::kKStages;
            const int k0 = tile_at(u.k, j) * kBlockN, here = page;
            if (j + 1 < u.s1) page = pages.look_up(p, at, dead, tile_at(u.k, j + 1) * kBlockN);  // ahead of its use
            if (it >= S::kKStages &&
                !(ok = ptx::warp_all(ptx::bar_wait(bar(S::kKEmpty + stage), ((it / S::kKStages) - 1) & 1, abort_flag,
                                     p.timeout_ns))))
                break;
            const uint32_t dst = sbase + S::kOffK + stage * S::kTileBytes;
            if (p.log2_bs < 3) {
                copy_small_pages<D>(p, at, dead, k0, p.k, dst);
                if (leader) ptx::bar_arrive(bar(S::kKFull + stage));
            } else {
                if (leader) ptx::bar_arrive_expect_tx(bar(S::kKFull + stage), S::kTileBytes);
                __syncwarp();
                pages.load<D>(p, at, dead, k0, here, tk, dst, bar(S::kKFull + stage));
                __syncwarp();
            }
            if (wi > 0 && j == u.s0 && !(ok = load_q())) break;
        }
        if (!ok) break;
        ++wi;
    }
    // Never leave with copies in flight (bounded, even after an abort).
    for (uint32_t s = 0; s < S::kKStages && s < it; ++s) {
        const uint32_t last = (it - 1) - ((it - 1 - s) % S::kKStages);
        ptx::bar_wait(bar(S::kKFull + s), (last / S::kKStages) & 1, nullptr, p.timeout_ns);
    }
    if (nq > 0) ptx::bar_wait(bar(S::kQFull), (nq - 1) & 1, nullptr, p.timeout_ns);
}

template <int D>
__device__ void producer_v(const CUtensorMap *tv, const ChunkParams &p, uint32_t sbase, const volatile Run *run,
                           volatile int *abort_flag) {
    using S = FwdShape<D>;
    const uint32_t bars = sbase + S::kOffBar;
    auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
    const bool leader = ptx::elect_one();
    const Pages pages(p);
    // (test support: the CTA with the first unit's first step)
    const bool first = blockIdx.x * run->per <= kStart && (blockIdx.x + 1) * run->per > kStart;
    uint32_t it = 0;
    uint32_t cuts = 0, cut_done = 0;  // tiles with rows to clear: loaded, landed
    bool ok = true;
    Walk walk;
    walk.start(p, run);
    Part u;
    while (ok && walk.next(p, u)) {
        if (u.s1 == u.s0) continue;
        const Dead dead(p, u.s);
        const Head at{u.b, u.hk, u.s.L};
        int page = pages.look_up(p, at, dead, tile_at(u.k, u.s0) * kBlockN);
        for (int j = u.s0; j < u.s1; ++j, ++it) {
            if (it == 1 && !(ok = ptx::warp_all(ptx::bar_wait(bar(S::kFirstQ), 0, abort_flag, p.timeout_ns)))) break;
            const uint32_t stage = it % S::kVStages;
            const int k0 = tile_at(u.k, j) * kBlockN, here = page;
            if (j + 1 < u.s1) page = pages.look_up(p, at, dead, tile_at(u.k, j + 1) * kBlockN);
            if (it >= S::kVStages &&
                !(ok = ptx::warp_all(ptx::bar_wait(bar(S::kVEmpty + stage), ((it / S::kVStages) - 1) & 1, abort_flag,
                                     p.timeout_ns))))
                break;
            const uint32_t dst = sbase + S::kOffV + stage * S::kTileBytes, full = bar(S::kVFull + stage);
            if (withheld(p.withhold, it, first)) continue;
            if (p.log2_bs < 3) {
                copy_small_pages<D>(p, at, dead, k0, p.v, dst);
                if (leader) ptx::bar_arrive(full);
                continue;
            }
            // Rows of a page that nobody sees may hold anything. Their weights
            // are zero, but 0 x NaN is not, so they are cleared before the tile
            // is handed on.
            const int end = u.s.L - k0;
            const bool cut = end < kBlockN || dead.any(k0, k0 + kBlockN);
            const uint32_t lands = cut ? bar(S::kVCut) : full;
            if (leader) ptx::bar_arrive_expect_tx(lands, S::kTileBytes);
            __syncwarp();
            pages.load<D>(p, at, dead, k0, here, tv, dst, lands);
            __syncwarp();
            if (cut) {
                if (!(ok = ptx::warp_all(ptx::bar_wait(lands, cuts++ & 1, abort_flag, p.timeout_ns)))) break;
                ++cut_done;
                if (end < kBlockN) ptx::zero_rows(dst, S::kColBlocks, kBlockN, end, kBlockN);
                const int z0 = max(dead.dead0 - k0, 0), z1 = min(dead.dead1 - k0, kBlockN);
                if (z0 < z1) ptx::zero_rows(dst, S::kColBlocks, kBlockN, z0, z1);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (leader) ptx::bar_arrive(full);
            }
        }
    }
    if (cuts > cut_done) ptx::bar_wait(bar(S::kVCut), (cuts - 1) & 1, nullptr, p.timeout_ns);
    for (uint32_t s = 0; s < S::kVStages && s < it; ++s) {
        const uint32_t last = (it - 1) - ((it - 1 - s) % S::kVStages);
        ptx::bar_wait(bar(S::kVFull + s), (last / S::kVStages) & 1, nullptr, p.timeout_ns);
    }
}

template <int D, bool BF16>
__device__ void mma(const ChunkParams &p, uint32_t sbase, uint32_t tmem, const volatile Run *run,
                    volatile int *abort_flag) {
    using S = FwdShape<D>;
    constexpr uint32_t kIdescQK = ptx::idesc_f16(BF16, kBlockM, kBlockN, false);
    constexpr uint32_t kIdescPV = ptx::idesc_f16(BF16, kBlockM, D, true);
    const uint32_t bars = sbase + S::kOffBar;
    auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
    const bool leader = ptx::elect_one();
    const uint64_t dq0 = ptx::smem_desc_sw128(sbase + S::kOffQ, 16, 1024);
    const uint64_t dk0 = ptx::smem_desc_sw128(sbase + S::kOffK, 16, 1024);
    const uint64_t dv0 = ptx::smem_desc_sw128(sbase + S::kOffV, S::kBlockBytes, 1024);
    constexpr uint64_t kTile16 = S::kTileBytes >> 4;

    // products as in the packed forward
    auto issue_qk = [&](int t, uint32_t stage) {
        const uint64_t qd = dq0 + static_cast<uint64_t>(t) * kTile16, kd = dk0 + static_cast<uint64_t>(stage) * kTile16;
        const uint32_t dst = tmem + S::kTmemS + t * 128;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            constexpr uint64_t kBlock16 = S::kBlockBytes >> 4;
            const uint64_t off = (kk / 4) * kBlock16 + (kk % 4) * 2;
            ptx::mma_ss(dst, qd + off, kd + off, kIdescQK, kk > 0);
        }
    };
    auto issue_pv = [&](int t, uint32_t stage, bool accumulate, int half) {
        const uint64_t vd = dv0 + static_cast<uint64_t>(stage) * kTile16;
        const uint32_t dst = tmem + S::kTmemO + t * D, pa = tmem + S::kTmemS + t * 128;
#pragma unroll
        for (int k4 = 0; k4 < kBlockN / 32; ++k4) {
            const int kk = half * (kBlockN / 32) + k4;
            ptx::mma_ts(dst, pa + kk * 8, vd + kk * (2048 >> 4), kIdescPV, (accumulate || kk > 0) ? 1u : 0u);
        }
    };

    uint32_t it = 0, wi = 0;   // K/V tiles consumed, parts consumed
    uint32_t cnt[2] = {0, 0};  // PV steps issued per query tile
    bool ok = true;
    Walk walk;
    walk.start(p, run);
    Part u;
    while (ok && walk.next(p, u)) {
        const int n = u.s1 - u.s0;
        if (n == 0) continue;
        const int total[2] = {visited(u.k, 0, u.s0, u.s1), visited(u.k, 1, u.s0, u.s1)};
        if (!(ok = ptx::warp_all(ptx::bar_wait(bar(S::kQFull), wi & 1, abort_flag, p.timeout_ns)))) break;
        if (wi == 0 && leader) ptx::bar_arrive(bar(S::kFirstQ));
        {
            const uint32_t ks = it % S::kKStages;
            if (!(ok = ptx::warp_all(ptx::bar_wait(bar(S::kKFull + ks), (it / S::kKStages) & 1, abort_flag, p.timeout_ns))))
                break;
            ptx::tc_fence_after();
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (!visits(u.k, t, u.s0)) continue;
                if (leader) {
                    issue_qk(t, ks);
                    ptx::mma_commit(bar(S::kSFull + t));
                }
            }
            if (leader) ptx::mma_commit(bar(S::kKEmpty + ks));
            if (n == 1 && leader) ptx::mma_commit(bar(S::kQEmpty));
        }
        int done[2] = {0, 0};
        for (int j = 0; j < n && ok; ++j) {
            const uint32_t itj = it + j;
            const uint32_t vs = itj % S::kVStages;
            const uint32_t kn = (itj + 1) % S::kKStages;
            bool v_ready = false, k_next_used = false;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (visits(u.k, t, u.s0 + j)) {
                    if (!(ok = ptx::warp_all(ptx::bar_wait(bar(S::kPFull + t), cnt[t] & 1, abort_flag, p.timeout_ns))))
                        break;
                    if (!v_ready) {
                        if (!(ok = ptx::warp_all(ptx::bar_wait(bar(S::kVFull + vs), (itj / S::kVStages) & 1, abort_flag,
                                                 p.timeout_ns))))
                            break;
                        v_ready = true;
                    }
                    ptx::tc_fence_after();
                    if (leader) issue_pv(t, vs, done[t] > 0, 0);
                    if (!(ok = ptx::warp_all(ptx::bar_wait(bar(S::kPFull2 + t), cnt[t] & 1, abort_flag, p.timeout_ns))))
                        break;
                    ptx::tc_fence_after();
                    if (leader) {
                        issue_pv(t, vs, true, 1);
                        if (done[t] + 1 == total[t]) ptx::mma_commit(bar(S::kODone + t));
                    }
                    ++cnt[t];
                    ++done[t];
                }
                if (j + 1 < n && visits(u.k, t, u.s0 + j + 1)) {
                    if (!k_next_used) {
                        if (!(ok = ptx::warp_all(ptx::bar_wait(bar(S::kKFull + kn), ((itj + 1) / S::kKStages) & 1, abort_flag,
                                                 p.timeout_ns))))
                            break;
                        k_next_used = true;
                    }
                    ptx::tc_fence_after();
                    if (leader) {
                        issue_qk(t, kn);
                        ptx::mma_commit(bar(S::kSFull + t));
                    }
                }
            }
            if (!ok) break;
            if (leader) {
                ptx::mma_commit(bar(S::kVEmpty + vs));
                if (k_next_used) ptx::mma_commit(bar(S::kKEmpty + kn));
                if (j + 2 == n) ptx::mma_commit(bar(S::kQEmpty));
            }
        }
        if (!ok) break;
        it += n;
        ++wi;
    }
    if (leader) ptx::mma_commit(bar(S::kTeardown));
    __syncwarp();
    ptx::bar_wait(bar(S::kTeardown), 0, nullptr, p.timeout_ns);
}

template <int D, bool BF16>
__device__ void softmax(const ChunkParams &p, uint32_t sbase, uint32_t tmem, int t, int wq, int lane,
                        Shared *sh, volatile int *abort_flag) {
    using S = FwdShape<D>;
    const uint32_t bars = sbase + S::kOffBar;
    auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
    const int row = wq * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_base + S::kTmemS + t * 128;
    const uint32_t tO = tmem + lane_base + S::kTmemO + t * D;
    const float scale_log2 = p.scale_log2;
    const uint64_t stream_pol = ptx::l2_policy_evict_first();
    uint32_t cnt = 0, items = 0;
    bool ok = true;
    Kept *kept = sh->kept + 4 * t + wq;
    if (lane == 0) kept->walk.start(p, &sh->run);
    __syncwarp();
    while (ok) {
        // the key tiles of this part that the query tile visits: [x, x1), then [x2, x3)
        int x, x1, x2, x3, first, behind;
        {
            Walk walk = kept->walk;
            Part u;
            if (!walk.next(p, u)) break;
            auto mine = [&](const int (&v)[2]) { return t == 0 ? v[0] : v[1]; };
            const int up = u.k.lo - u.k.ns, ntok = mine(u.k.ntok);
            x = u.s0;
            x1 = min(u.s1, mine(u.k.sink));
            x2 = max(max(mine(u.k.wlo), u.k.ns), u.s0 + up);
            x3 = min(mine(u.k.hi), u.s1 + up);
            if (x >= x1) x1 = x = x2;  // no first run
            first = u.s.L - u.s.Lq + mine(u.k.tok);  // the tile's first position
            behind = p.window > 0 ? first + ntok - 1 - p.window : -1;  // the last key behind its last window
            __syncwarp();
            if (lane == 0) {
                kept->walk = walk;
                kept->tok0 = u.s.q0 + mine(u.k.tok);
                kept->ntok = ntok;
                kept->h0 = u.hk * p.group;
                kept->dest = u.whole ? -1 : u.slot;
            }
            __syncwarp();
            if (ntok == 0) continue;
        }
        const int pos = first + row / p.group;
        float m_used = -CUDART_INF_F;
        float l = 0.f;
        int mine = 0;  // steps taken
        for (;; ++x) {
            if (x == x1) x = x2;
            if (x >= x3 && x >= x1) break;
            ok = ptx::bar_wait(bar(S::kSFull + t), cnt & 1, abort_flag, p.timeout_ns);
            if (!__all_sync(kFull, ok)) { ok = false; break; }
            ptx::tc_fence_after();
            // the row sees the columns c < lim, but with a window not those with sk <= c < wl
            const int k0 = x * kBlockN;
            const bool need_mask = k0 + kBlockN - 1 > first;
            const bool need_lo = k0 + kBlockN > p.sinks && k0 <= behind;
            uint32_t s[4][32];
            float mx4[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) ptx::tmem_ld32_max(tS + 32 * c, s[c], mx4[c]);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                ptx::reg_fence(s[c]);
                asm volatile("" : "+f"(mx4[c]));
            }
            if (need_mask || need_lo) {
                // the columns c < x as bits of chunk b: its low x - 32 b
                auto below = [](int x, int b) -> uint32_t {
                    const int n = min(max(x - 32 * b, 0), 32);
                    return static_cast<uint32_t>((1ull << n) - 1);
                };
                const int lim = pos + 1 - k0, wl = p.window > 0 ? pos - p.window + 1 - k0 : 0, sk = p.sinks - k0;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const uint32_t seen = below(lim, b) & (below(sk, b) | ~below(wl, b));
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!(seen & (1u << i))) s[b][i] = 0xff800000u;  // -inf
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) mx4[c] = -CUDART_INF_F;
#pragma unroll
                for (int c = 0; c < kBlockN; c += 2)
                    mx4[(c / 2) % 4] = ptx::fmax3(mx4[(c / 2) % 4], __uint_as_float(s[c / 32][c % 32]),
                                                  __uint_as_float(s[(c + 1) / 32][(c + 1) % 32]));
            }
            const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
            const float m_cand = mx * scale_log2;
            const bool need = m_cand > m_used + kRescaleThreshold;
            float alpha = 1.f;
            if (need) {
                alpha = ptx::ex2(m_used - m_cand);
                m_used = m_cand;
            }
            l *= alpha;
            const float m_sub = (m_used == -CUDART_INF_F) ? 0.f : m_used;
            const uint64_t scale2 = ptx::pk2(scale_log2, scale_log2);
            const uint64_t negm2 = ptx::pk2(-m_sub, -m_sub);
            uint64_t sum2[2] = {ptx::pk2(0.f, 0.f), ptx::pk2(0.f, 0.f)};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t pk[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int c = 64 * h + 2 * i;
                    const uint64_t x = ptx::ffma2(ptx::pk2(__uint_as_float(s[c / 32][c % 32]),
                                                           __uint_as_float(s[(c + 1) / 32][(c + 1) % 32])),
                                                  scale2, negm2);
                    float x0, x1;
                    ptx::upk2(x, x0, x1);
                    const float e0 = ptx::ex2(x0), e1 = ptx::ex2(x1);
                    sum2[i % 2] = ptx::fadd2(sum2[i % 2], ptx::pk2(e0, e1));
                    pk[i] = ptx::pack2<BF16>(e0, e1);
                }
                ptx::tmem_st32(tS + 32 * h, pk);
                if (h == 0 && mine > 0 && __any_sync(kFull, need)) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        ptx::tmem_ld32(tO + c * 32, o);
                        ptx::tmem_ld_wait();
                        ptx::reg_fence(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        ptx::tmem_st32(tO + c * 32, o);
                    }
                }
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::bar_arrive(bar((h == 0 ? S::kPFull : S::kPFull2) + t));
            }
            {
                float a0, a1, b0, b1;
                ptx::upk2(sum2[0], a0, a1);
                ptx::upk2(sum2[1], b0, b1);
                l += (a0 + a1) + (b0 + b1);
            }
            ++cnt;
            ++mine;
        }
        if (!ok) break;

        if (mine > 0) {
            ok = ptx::bar_wait(bar(S::kODone + t), items & 1, abort_flag, p.timeout_ns);
            if (!__all_sync(kFull, ok)) { ok = false; break; }
            ptx::tc_fence_after();
            ++items;
        }
        const volatile Kept *end = kept;
        const int dest = end->dest, token = row / p.group;  // token within the tile
        const bool row_valid = token < end->ntok;           // (it has at most tile_tokens)
        uint32_t o[D / 32][32];
        if (mine > 0) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) ptx::tmem_ld32(tO + c * 32, o[c]);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < D / 32; ++c) ptx::reg_fence(o[c]);
        } else {
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i) o[c][i] = 0u;
        }
        if (dest >= 0) {
            // a part: m, l and O as they are, four columns of all rows after another, so
            // that a warp's stores are whole lines
            if (row_valid) {
                const size_t part = 2 * blockIdx.x + dest, r = t * kBlockM + row;
                float4 *dst = reinterpret_cast<float4 *>(p.o_part) + part * (D / 4) * p.part_rows + r;
#pragma unroll
                for (int c = 0; c < D; c += 4)
                    dst[c / 4 * p.part_rows] =
                        make_float4(__uint_as_float(o[c / 32][c % 32]), __uint_as_float(o[c / 32][c % 32 + 1]),
                                    __uint_as_float(o[c / 32][c % 32 + 2]), __uint_as_float(o[c / 32][c % 32 + 3]));
                p.ml_part[part * p.part_rows + r] = make_float2(m_used, l);
            }
            continue;
        }
        // O / l in the input dtype, LSE = (m + log2 l) * ln 2
        const float inv_l = l == 0.f ? 0.f : 1.f / l;
        const float lse = l == 0.f ? -CUDART_INF_F : (m_used + __log2f(l)) * 0.69314718055994531f;
        if (row_valid) {
            const size_t tok = static_cast<size_t>(end->tok0) + token, h = end->h0 + row - token * p.group;
            uint16_t *orow = static_cast<uint16_t *>(p.o) + (tok * p.H + h) * D;
            const bool v8 = (reinterpret_cast<uintptr_t>(p.o) & 31) == 0;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    pk[i] = ptx::pack2<BF16>(__uint_as_float(o[c][2 * i]) * inv_l, __uint_as_float(o[c][2 * i + 1]) * inv_l);
                uint4 *dst = reinterpret_cast<uint4 *>(orow + c * 32);
                if (v8) {
                    ptx::st_global_v8_hint(dst, pk, stream_pol);
                    ptx::st_global_v8_hint(dst + 2, pk + 8, stream_pol);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) dst[i] = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
                }
            }
            p.lse[h * p.total_q + tok] = lse;
        }
    }
}

// ----------------------------------------------------------------- kernels --

template <int D, bool BF16>
__global__ void __launch_bounds__(kFwdThreads, 1)
    fa_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const ChunkParams p) {
    using S = FwdShape<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = ptx::smem_addr(smem);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + S::kOffMisc + 4);
    Shared *sh = reinterpret_cast<Shared *>(smem + S::kOffSched);
    Run *run = &sh->run;
    static_assert(sizeof(Shared) <= kSchedInts * 4 && kPlanBytes <= S::kOffBar, "shared memory budget");
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    // the plan's scratch lies where the tiles go
    plan(p, Units{p}, run, smem);
    if (warp == 1) {
        if (lane == 0) {
            const uint32_t bars = sbase + S::kOffBar;
            for (int i = 0; i < S::kNumBars; ++i) {
                const bool p_full = i >= S::kPFull && i < S::kODone;
                ptx::bar_init(bars + 8u * i, p_full ? kBlockM / 32 : 1u);
            }
            *abort_flag = 0;
            ptx::bar_init_fence();
        }
        __syncwarp();
        ptx::tmem_alloc(ptx::smem_addr(tmem_slot), S::kTmemCols);
        ptx::tmem_relinquish();
    } else if (warp == 2 && lane == 0) {
        ptx::prefetch_tmap(&tm_q);
        ptx::prefetch_tmap(&tm_k);
        ptx::prefetch_tmap(&tm_v);
    }
    ptx::fence_proxy_async_smem();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        producer_qk<D>(&tm_q, &tm_k, p, sbase, run, abort_flag);
    } else if (warp == 1) {
        mma<D, BF16>(p, sbase, tmem, run, abort_flag);
    } else if (warp == 2) {
        producer_v<D>(&tm_v, p, sbase, run, abort_flag);
    } else if (warp == 3) {
        // the unit that starts here and ends in a later CTA's run, for the joining launch
        Walk walk;
        walk.start(p, run);
        Part u;
        int4 rec = make_int4(0, 0, 0, 0);
        while (walk.next(p, u))
            if (u.parts > 0)
                rec = make_int4(u.s.q0 + u.k.tok[0], u.k.ntok[0] + u.k.ntok[1], u.hk * p.group, 2 * u.parts + u.slot);
        if (lane == 0) p.records[blockIdx.x] = rec;
    } else {
        softmax<D, BF16>(p, sbase, tmem, (warp - 4) / 4, warp % 4, lane, sh, abort_flag);
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, S::kTmemCols);
    }
    if (threadIdx.x == 0 && *abort_flag) atomicExch(p.err, kDeviceErrTimeout);
}

constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 32;  // of a unit, per CTA

// Joins the parts of units that fell into several runs: CTA x for the unit that
// started in run x, if any. A lane has a row, a warp D / 8 of its columns (reads are
// whole lines); the rows go out through shared memory. Where there are fewer rows
// than lanes, lanes share out the parts of a row: one token of 8 heads on one key head,
// 131000 keys in some 150 parts, 45 us in place of 93.
template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) fa_chunk_join_kernel(const ChunkParams p) {
    constexpr int kWarps = kJoinThreads / 32, kQuads = D / 4 / kWarps;  // of four columns, a warp
    __shared__ uint2 tile[kJoinRows][D / 4 + 1];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int4 rec = __ldcg(p.records + blockIdx.x);  // first packed row, tokens, first head, 2 parts + slot of the first
    const int parts = min(rec.w / 2, static_cast<int>(gridDim.x - blockIdx.x)), slot = rec.w & 1;
    if (parts == 0) return;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    // token (of the unit) and head (of the group) of row r, -1 where it is none
    auto where = [&](int r, int &head) {
        const int token = r % kBlockM / p.group, tok = r / kBlockM * p.tile_tokens + token;
        head = r % kBlockM - token * p.group;
        return r < p.part_rows && token < p.tile_tokens && tok < rec.y ? tok : -1;
    };
    const int rows = p.part_rows >= 32 ? 32 : 1 << (32 - __clz(p.part_rows - 1)), slices = 32 / rows, slice = lane / rows;
    const int row = blockIdx.y * kJoinRows + lane % rows;
    int head;
    const int tok = where(row, head), end = tok >= 0 ? parts : 0;
    // part 0 is in the slot it was given, later ones in the first of their CTAs
    auto at = [&](int x) { return static_cast<size_t>(2 * (blockIdx.x + x) + (x == 0 ? slot : 0)); };
    float m = -CUDART_INF_F, l = 0.f;
#pragma unroll 4
    for (int x = slice; x < end; x += slices) m = fmaxf(m, __ldcg(p.ml_part + at(x) * p.part_rows + row).x);
    for (int off = rows; off < 32; off *= 2) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
    float4 o[kQuads];
#pragma unroll
    for (int i = 0; i < kQuads; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int x = slice; x < end; x += slices) {
        const float2 ml = __ldcg(p.ml_part + at(x) * p.part_rows + row);
        const float4 *v = reinterpret_cast<const float4 *>(p.o_part) + (at(x) * (D / 4) + warp * kQuads) * p.part_rows + row;
        const float f = ml.x == -CUDART_INF_F ? 0.f : ptx::ex2(ml.x - m);
        l = fmaf(ml.y, f, l);
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
            const float4 y = __ldcg(v + i * p.part_rows);
            o[i].x = fmaf(y.x, f, o[i].x);
            o[i].y = fmaf(y.y, f, o[i].y);
            o[i].z = fmaf(y.z, f, o[i].z);
            o[i].w = fmaf(y.w, f, o[i].w);
        }
    }
    for (int off = rows; off < 32; off *= 2) {
        auto add = [&](float &a) { a += __shfl_xor_sync(kFull, a, off); };
        add(l);
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
            add(o[i].x);
            add(o[i].y);
            add(o[i].z);
            add(o[i].w);
        }
    }
    if (tok >= 0 && slice == 0) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
            tile[lane][warp * kQuads + i] = make_uint2(ptx::pack2<BF16>(o[i].x * inv, o[i].y * inv),
                                                       ptx::pack2<BF16>(o[i].z * inv, o[i].w * inv));
        if (warp == 0)
            p.lse[static_cast<size_t>(rec.z + head) * p.total_q + rec.x + tok] =
                l == 0.f ? -CUDART_INF_F : (m + __log2f(l)) * 0.69314718055994531f;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kJoinRows * (D / 4); i += kJoinThreads) {
        const int r = i / (D / 4), c = i % (D / 4), t = where(blockIdx.y * kJoinRows + r, head);
        if (t >= 0)
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.o) +
                                       (static_cast<size_t>(rec.x + t) * p.H + rec.z + head) * D + 4 * c) = tile[r][c];
    }
}

template <int D, bool BF16>
cudaError_t launch_t(const CUtensorMap *maps, const ChunkParams &p, int grid, cudaStream_t st) {
    static std::atomic<unsigned long long> done{0};
    auto kern = fa_chunk_kernel<D, BF16>;
    constexpr int kSmem = FwdShape<D>::kSmemBytes;
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(kern), kSmem, done);
    if (e != cudaSuccess) return e;
    // Early where there is a unit for an SM at most (two short chunks 16.7 -> 14.5 us, 5
    // tokens of 16 sequences of up to 8192 keys 79 -> 78). With more units it costs: the
    // CTAs then lie where SMs came free first, not in their order (16 chunks of 1 to 512
    // tokens 292 -> 303, 2048 tokens behind 30000 keys 627 -> 650).
    const long long units = (static_cast<long long>(p.total_q / (2 * p.tile_tokens)) + p.B) * p.Hkv;
    e = launch_early(kern, dim3(static_cast<unsigned>(grid)), kFwdThreads, kSmem, st, units <= grid, maps[0], maps[1],
                     maps[2], p);
    if (e != cudaSuccess) return e;
    const dim3 join(static_cast<unsigned>(grid), static_cast<unsigned>((p.part_rows + kJoinRows - 1) / kJoinRows));
    return launch_early(fa_chunk_join_kernel<D, BF16>, join, kJoinThreads, 0, st, true, p);
}

}  // namespace chunk
}  // namespace fa
