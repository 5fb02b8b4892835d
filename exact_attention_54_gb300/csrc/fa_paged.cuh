// Shared by the kernels that take chunks of queries over a paged 16-bit cache
// (fa_chunk.cuh, fa_weights.cu): the cut of the work into equal runs, made by
// every CTA from the lengths on the device, and key tiles out of pages.
#pragma once

#include <climits>

#include "fa_fwd_kernel.cuh"

namespace fa {
namespace paged {

constexpr int kPlanEntries = 4096;  // the plan's table: sums over a sequence, or over several if there are more
constexpr int kSerialUnits = 16;    // units of a sequence that a thread adds up, rather than a warp,
constexpr int kPlanLong = 4096;     // where a sequence has more and there are no more than this many such
constexpr int kPlanSeqs = 512;      // sequences that are not loaded again for the CTA's place
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

constexpr int kPlanBytes = 8 * (kPlanEntries + 1) + 4 * (kPlanLong + 1) + static_cast<int>(sizeof(Seq)) * kPlanSeqs;

// A CTA's run of the laid-out units, in shared memory.
struct Run {
    long long len;     // cost units, 0: no work
    long long per;     // of every CTA but the last; 0: nothing is computed
    int b, hk, unit;   // the unit it starts in,
    int off;           // and where,
    Seq s;             // its sequence
};

// ------------------------------------------------------------------- plan --

// a / b; a 64-bit division costs some 500 clocks of latency.
__device__ __forceinline__ unsigned long long divide(unsigned long long a, unsigned long long b) {
    if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
    return a / b;
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    return v;
}

// Cost of one key head of a sequence's n units. Units [flat.x, flat.y) cost the
// same, the others are added up: by `lanes` threads, of which this is `lane`.
template <class Units>
__device__ __forceinline__ unsigned long long seq_cost(const Units &units, const Seq &s, int n, int2 flat, int lane,
                                                       int lanes) {
    unsigned long long c = 0;
    for (int i = lane; i < flat.x; i += lanes) c += units.cost(s, i);
    for (int i = flat.y + lane; i < n; i += lanes) c += units.cost(s, i);
    if (lane == 0 && flat.y > flat.x) c += static_cast<unsigned long long>(flat.y - flat.x) * units.cost(s, flat.x);
    return c;
}

// This CTA's run into `run`; scratch: kPlanBytes of shared memory. units:
// count(s) units of each key head of a sequence, cost(s, i) of the i-th, flat(s, n)
// a range of them that cost the same. The whole CTA calls it, and synchronises
// before it reads `run`; all warps but the first return while that one looks for
// the CTA's place, so what else a kernel sets up comes behind this. It stands between
// a launch and its first load (with one warp adding up all units: 8 us for 16
// sequences of up to 8192 keys), so a thread takes a sequence with few units to add
// up, warps share out the others, and nothing divides in 64 bits without need.
template <class Units>
__device__ void plan(const PagedParams &p, const Units units, Run *run, void *scratch) {
    unsigned long long *prefix = static_cast<unsigned long long *>(scratch);
    int *many = reinterpret_cast<int *>(prefix + kPlanEntries + 1), *n_many = many + kPlanLong;
    Seq *seqs = reinterpret_cast<Seq *>(n_many + 1);
    const int each = (p.B + kPlanEntries - 1) / kPlanEntries, entries = (p.B + each - 1) / each;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    // (a thread's first loads are ahead of the scratch's clearing)
    int q0 = 0, q1 = 0, keys = 0;
    if (threadIdx.x < p.B) {
        q0 = p.cu_q[threadIdx.x];
        q1 = p.cu_q[threadIdx.x + 1];
        keys = p.seq_lens[threadIdx.x];
    }
    if (threadIdx.x == 0) *n_many = 0;
    for (int i = threadIdx.x; i < entries; i += blockDim.x) prefix[i + 1] = 0;
    __syncthreads();
    bool bad = false;
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
        if (b >= blockDim.x) {
            q0 = p.cu_q[b];
            q1 = p.cu_q[b + 1];
            keys = p.seq_lens[b];
        }
        const Seq s{q0, q1 - q0, min(max(keys, 0), p.max_blocks << p.log2_bs)};
        if (q0 < 0 || q1 < q0 || q1 > p.total_q || q1 - q0 > p.max_q) {
            bad = true;
            continue;
        }
        if (b < kPlanSeqs) seqs[b] = s;
        const int n = units.count(s);
        const int2 flat = units.flat(s, n);
        const int at = n - (flat.y - flat.x) > kSerialUnits ? atomicAdd(n_many, 1) : kPlanLong;
        if (at < kPlanLong) {
            many[at] = b;
        } else if (n > 0) {
            const unsigned long long c = seq_cost(units, s, n, flat, 0, 1);
            if (each == 1) prefix[b + 1] = c;
            else if (c > 0) atomicAdd(&prefix[b / each + 1], c);
        }
    }
    bad = __syncthreads_or(bad) != 0;
    if (bad) {
        if (threadIdx.x == 0) {
            atomicExch(p.err, kDeviceErrSeqLens);
            run->len = run->per = 0;
        }
        return;
    }
    for (int i = warp; i < min(*n_many, kPlanLong); i += blockDim.x / 32) {
        const Seq s = load_seq(p, many[i]);
        const int n = units.count(s);
        const unsigned long long c = warp_sum(seq_cost(units, s, n, units.flat(s, n), lane, 32));
        if (lane == 0 && c > 0) atomicAdd(&prefix[many[i] / each + 1], c);
    }
    __syncthreads();
    if (warp != 0) return;
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
    const long long per = max(static_cast<long long>(divide(total + gridDim.x - 1, gridDim.x)), 1LL);
    const long long at = min(static_cast<long long>(blockIdx.x) * per, total);
    const long long len = min(per, total - at);
    Run r{len, per, 0, 0, 0, 0, Seq{0, 0, 0}};
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
        int2 flat{};
        unsigned long long c = 0;
        for (r.b = lo * each;; ++r.b) {
            s = r.b < kPlanSeqs ? seqs[r.b] : load_seq(p, r.b);
            n = units.count(s);
            flat = units.flat(s, n);
            c = each == 1 ? prefix[r.b + 1] - prefix[r.b] : warp_sum(seq_cost(units, s, n, flat, lane, 32));
            if (x < c * p.Hkv || r.b + 1 >= p.B) break;
            x -= c * p.Hkv;
        }
        r.s = s;
        r.hk = static_cast<int>(divide(x, c));
        x -= c * r.hk;
        // the unit whose share holds x: of [i0, i1), one by one
        auto among = [&](int i0, int i1) {
            for (; i0 < i1; i0 += 32) {
                const unsigned long long v = i0 + lane < i1 ? units.cost(s, i0 + lane) : 0;
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
                    return true;
                }
                x -= __shfl_sync(kFull, upto, 31);
            }
            return false;
        };
        if (!among(0, flat.x)) {
            const unsigned one = flat.y > flat.x ? units.cost(s, flat.x) : 0;
            const unsigned long long all = static_cast<unsigned long long>(flat.y - flat.x) * one;
            if (x < all) {
                const unsigned at = static_cast<unsigned>(divide(x, one));
                r.unit = flat.x + static_cast<int>(at);
                r.off = static_cast<int>(x - static_cast<unsigned long long>(at) * one);
            } else {
                x -= all;
                among(flat.y, n);
            }
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
