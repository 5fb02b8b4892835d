// Shared by the kernels that take chunks of queries over a paged 16-bit cache
// (fa_chunk.cuh, fa_weights.cu): the cut of the work into equal runs, made by
// every CTA from the lengths on the device, and key tiles out of pages.
#pragma once

#include <climits>

#include "fa_fwd_kernel.cuh"

namespace fa {
namespace paged {

constexpr int kPlanEntries = 4096;  // the plan's table: sums over a sequence, or over several if there are more
constexpr int kSerialUnits = 16;    // a thread sums the units of a sequence with up to this many, a warp longer ones
constexpr unsigned kFull = 0xffffffffu;

// Sequence b's chunk: its rows in the packed queries, its keys.
struct Seq {
    int q0, Lq, L;
};

__device__ __forceinline__ Seq load_seq(const PagedParams &p, int b) {
    Seq s;
    s.q0 = p.cu_q[b];
    s.Lq = p.cu_q[b + 1] - s.q0;
    s.L = min(max(p.seq_lens[b], 0), p.max_blocks << p.log2_bs);
    return s;
}

// A CTA's run of the laid-out units, in shared memory.
struct Run {
    long long len;     // cost units, 0: no work
    long long per;     // of every CTA but the last
    int b, hk, unit;   // the unit it starts in,
    int off;           // and where
};

// ------------------------------------------------------------------- plan --

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    return v;
}

// Cost of one key head of a sequence's n units; the whole warp calls it.
template <class Units>
__device__ __forceinline__ unsigned long long seq_cost(const Units &units, const Seq &s, int n) {
    unsigned long long c = 0;
    for (int i = threadIdx.x % 32; i < n; i += 32) c += units.cost(s, i);
    return warp_sum(c);
}

// This CTA's run into `run`; `prefix` is scratch of kPlanEntries + 1 sums.
// units: count(s) units of each key head of a sequence, cost(s, i) of the i-th.
// The whole CTA calls it, and synchronises before it reads `run`.
template <class Units>
__device__ void plan(const PagedParams &p, const Units units, Run *run, unsigned long long *prefix) {
    const int each = (p.B + kPlanEntries - 1) / kPlanEntries, entries = (p.B + each - 1) / each;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    for (int i = threadIdx.x; i < entries; i += blockDim.x) prefix[i + 1] = 0;
    __syncthreads();
    bool bad = false;
    for (int b0 = warp * 32; b0 < p.B; b0 += blockDim.x) {
        const int b = b0 + lane;
        Seq s{0, 0, 0};
        int n = 0;
        unsigned long long c = 0;
        if (b < p.B) {
            const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1];
            if (q0 < 0 || q1 < q0 || q1 > p.total_q || q1 - q0 > p.max_q) {
                bad = true;
            } else {
                s = load_seq(p, b);
                n = units.count(s);
                if (n <= kSerialUnits)
                    for (int i = 0; i < n; ++i) c += units.cost(s, i);
            }
        }
        unsigned more = __ballot_sync(kFull, n > kSerialUnits);
        while (more != 0) {
            const int l = __ffs(more) - 1;
            more &= more - 1;
            const Seq x{0, __shfl_sync(kFull, s.Lq, l), __shfl_sync(kFull, s.L, l)};
            const unsigned long long sum = seq_cost(units, x, __shfl_sync(kFull, n, l));
            if (lane == l) c = sum;
        }
        if (c > 0) atomicAdd(&prefix[b / each + 1], c);
    }
    bad = __syncthreads_or(bad) != 0;
    if (bad && threadIdx.x == 0) {
        atomicExch(p.err, kDeviceErrSeqLens);
        run->len = 0;
    }
    if (bad || warp != 0) return;
    // prefix sums of the entries; then this CTA's place among them
    const int mine = (entries + 31) / 32, e0 = lane * mine;
    unsigned long long sum = 0;
    for (int e = e0; e < min(e0 + mine, entries); ++e) sum += prefix[e + 1];
    unsigned long long before = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const unsigned long long v = __shfl_up_sync(kFull, before, off);
        if (lane >= off) before += v;
    }
    const long long total = static_cast<long long>(__shfl_sync(kFull, before, 31)) * p.Hkv;
    before -= sum;
    for (int e = e0; e < min(e0 + mine, entries); ++e) prefix[e + 1] = before += prefix[e + 1];
    if (lane == 0) prefix[0] = 0;
    __syncwarp();
    const long long per = max((total + gridDim.x - 1) / gridDim.x, static_cast<long long>(p.min_run));
    const long long at = min(static_cast<long long>(blockIdx.x) * per, total);
    const long long len = min(per, total - at);
    Run r{len, per, 0, 0, 0, 0};
    if (len > 0) {
        int lo = 0, hi = entries;  // the last entry that starts at or before `at`, and is not empty
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (static_cast<long long>(prefix[mid]) * p.Hkv <= at) lo = mid;
            else hi = mid;
        }
        unsigned long long x = static_cast<unsigned long long>(at) - prefix[lo] * p.Hkv;
        Seq s{};
        int n = 0;
        unsigned long long c = 0;
        for (r.b = lo * each;; ++r.b) {
            s = load_seq(p, r.b);
            n = units.count(s);
            c = seq_cost(units, s, n);
            if (x < c * p.Hkv || r.b + 1 >= p.B) break;
            x -= c * p.Hkv;
        }
        r.hk = static_cast<int>(x / c);
        x -= c * r.hk;
        // the unit whose share holds x
        for (int i0 = 0; i0 < n; i0 += 32) {
            const unsigned long long v = i0 + lane < n ? units.cost(s, i0 + lane) : 0;
            unsigned long long upto = v;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const unsigned long long y = __shfl_up_sync(kFull, upto, off);
                if (lane >= off) upto += y;
            }
            const unsigned here = __ballot_sync(kFull, x < upto);
            if (here != 0) {
                const int l = __ffs(here) - 1;
                r.unit = i0 + l;
                r.off = static_cast<int>(x - __shfl_sync(kFull, upto - v, l));
                break;
            }
            x -= __shfl_sync(kFull, upto, 31);
        }
    }
    if (lane == 0) *run = r;
}

// ------------------------------------------------------------------ loads --

// A key head of a sequence of L keys.
struct Head {
    int b, hk, L;
};

// Keys that no query of the chunk sees: from L on, and [dead0, dead1).
struct Dead {
    int dead0, dead1;
    __device__ __forceinline__ Dead(const PagedParams &p, const Seq &s) {
        dead0 = p.sinks;
        dead1 = p.window > 0 ? s.L - s.Lq - p.window + 1 : 0;
    }
    // all of [a, b)
    __device__ __forceinline__ bool all(int a, int b) const { return a >= dead0 && b <= dead1; }
    // any of [a, b)
    __device__ __forceinline__ bool any(int a, int b) const { return max(a, dead0) < min(b, dead1); }
};

// The pages of a key tile, one per lane (of the first kBlockN / span).
struct Pages {
    int span_log2;  // rows of a page within a tile
    int count;

    __device__ __forceinline__ Pages(const PagedParams &p) {
        span_log2 = min(p.log2_bs, 7);
        count = kBlockN >> span_log2;
    }
    // This lane's page of the tile from key k0 on: its number, -1 where no key
    // of it is seen (not looked up).
    __device__ __forceinline__ int look_up(const PagedParams &p, const Head &u, const Dead &d, int k0) const {
        const int lane = threadIdx.x % 32, key = k0 + (lane << span_log2);
        if (lane >= count || key >= u.L || d.all(key, min(key + (1 << span_log2), u.L))) return -1;
        return p.block_table[static_cast<size_t>(u.b) * p.max_blocks + (key >> p.log2_bs)];
    }
    // Its rows into the tile at `dst`, every lane its page; a page number that
    // does not exist is reported and stands for zeros, as do keys nobody sees.
    template <int D>
    __device__ __forceinline__ void load(const PagedParams &p, const Head &u, const Dead &d, int k0, int page,
                                         const CUtensorMap *tm, uint32_t dst, uint32_t bar) const {
        using S = FwdShape<D>;
        const int lane = threadIdx.x % 32, key = k0 + (lane << span_log2);
        if (lane >= count) return;
        const bool there = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_blocks);
        if (!there && key < u.L && !d.all(key, min(key + (1 << span_log2), u.L)))
            atomicExch(p.err, kDeviceErrBadIndex);
        const int z = there ? page * p.Hkv + u.hk : p.num_blocks * p.Hkv;
        const int y = key & ((1 << p.log2_bs) - 1);
#pragma unroll
        for (int c = 0; c < S::kColBlocks; ++c)
            ptx::tma_load_3d(dst + c * S::kBlockBytes + ((lane << span_log2) << 7), tm, bar, c * 64, y, z);
    }
};

// A tile from pages of less than 8 rows, by the whole warp: 16-byte pieces into
// the places that the swizzle gives them, zeros for keys nobody sees. Returns
// with the pieces landed and visible to the tensor core.
template <int D>
__device__ __forceinline__ void copy_small_pages(const PagedParams &p, const Head &u, const Dead &d, int k0,
                                                 const uint16_t *cache, uint32_t dst) {
    using S = FwdShape<D>;
    constexpr int kPieces = D / 8, kRows = 32 / kPieces;
    const int lane = threadIdx.x % 32, piece = lane % kPieces;
#pragma unroll 4
    for (int row = lane / kPieces; row < kBlockN; row += kRows) {
        const int key = k0 + row;
        const uint16_t *src = cache;
        uint32_t bytes = 0;
        if (key < u.L && !d.all(key, key + 1)) {
            const int page = p.block_table[static_cast<size_t>(u.b) * p.max_blocks + (key >> p.log2_bs)];
            if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_blocks)) {
                src += (((static_cast<long long>(page) * p.Hkv + u.hk) << p.log2_bs) + (key & ((1 << p.log2_bs) - 1))) *
                           D + piece * 8;
                bytes = 16;
            } else {
                atomicExch(p.err, kDeviceErrBadIndex);
            }
        }
        ptx::copy_async16(dst + (piece / 8) * S::kBlockBytes + row * 128 + (((piece % 8) ^ (row % 8)) << 4), src, bytes);
    }
    ptx::copy_async_wait_all();
    ptx::fence_proxy_async_smem();
    __syncwarp();
}

}  // namespace paged
}  // namespace fa
