// Eviction from a paged 16-bit cache by accumulated attention weight
// (fa_kv_evict): of each sequence and key head the first `sinks` keys, the last
// `recent` and the heaviest between them stay, in their order, in new pages.
//
// Two launches. Selection: a cluster of CTAs per (sequence, key head), as many as
// there are SMs for, each with a run of its keys, finds the weight of the last key
// that stays as an order statistic, digit by digit from the top (11, 11 and 10
// bits of the weight's bits, ordered as integers; the CTAs add up their counts
// through distributed shared memory), then writes the keys above it, and as many of
// the equal ones as there is room for, by prefix sums over the keys. The search works
// on the weights' order in shared memory, as far as it fits (behind that each digit reads
// the weights again); the weights themselves are read once more, to be written. Copy:
// lane groups of 16-byte pieces, page by table on both sides; a stream of 2 D bytes
// read and written per key and value.
//
// Bound: the copy by HBM; the selection by latency, of loads, of the cluster's barriers
// and of its counts (some 1,800 clocks each a digit). Four caches of 16384 to 32768 keys,
// 8 key heads, D = 128, down to 4096: 38 us, about 13 of them the selection; two caches
// of at most 777 keys 9 us.
#include <cooperative_groups.h>

#include "fa_launch.h"
#include "sm103_ptx.cuh"

namespace fa {
namespace evict {

constexpr int kThreads = 1024;
constexpr int kMaxCtas = 8;            // of a cluster (the portable size)
constexpr int kMaxCached = 44 * 1024;  // keys whose weights a CTA's shared memory holds
constexpr int kBins = 2048;
constexpr int kBatch = 8;  // loads of a thread in flight
constexpr unsigned kFull = 0xffffffffu;

// A weight's bits, ordered like the weights as unsigned integers: -0 is +0, a NaN is below everything.
__device__ __forceinline__ uint32_t order(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// Sum of v over this lane and those before it.
__device__ __forceinline__ uint32_t scan(uint32_t v) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(kFull, v, off);
        if (static_cast<int>(threadIdx.x % 32) >= off) v += y;
    }
    return v;
}

// Barriers cost a few hundred clocks each, so a digit takes two: the counts are
// there, and the sums over each warp's bins are; every warp then finds the digit
// for itself. The search ends where all keys of a digit stay, mostly after two. The
// keys that stay are written warp by warp, each over a run of keys. (Before: prefix
// sums of the whole CTA, 8 barriers a digit and 3 every 4096 keys, the others' counts
// one after another, always three digits: 22 us for the four caches above, 13 now.)
__global__ void __launch_bounds__(kThreads, 1) fa_kv_evict_select_kernel(const EvictParams p) {
    constexpr int kWarps = kThreads / 32, kOfWarp = kBins / kWarps;  // bins
    static_assert(kOfWarp == 64, "two bins a lane");
    extern __shared__ uint32_t cached[];  // the order of this CTA's first p.cached keys
    __shared__ uint32_t hist[3][kBins], sum[kBins], of_warp[3][kWarps];
    __shared__ uint2 counts[kWarps];  // of a warp's keys: above the last that stays, equal to it
    auto cluster = cooperative_groups::this_cluster();
    const int ctas = static_cast<int>(cluster.num_blocks()), cta = static_cast<int>(cluster.block_rank());
    const int tid = static_cast<int>(threadIdx.x), lane = tid % 32, warp = tid / 32;
    const int all = cta * kThreads + tid, step = ctas * kThreads;
    auto sync = [&] {
        if (ctas > 1) cluster.sync();
        else __syncthreads();
    };
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const size_t bh = blockIdx.x / ctas;
    const int b = static_cast<int>(bh / p.Hkv);
    const int width = p.max_blocks << p.log2_bs, new_width = p.new_max_blocks << p.log2_bs;
    const int L = min(max(p.seq_lens[b], 0), width), n = min(L, p.keep);
    const float *w = p.weights + bh * width;
    int *kept = p.kept + bh * p.keep;
    float *out = p.new_weights + bh * new_width;
    auto store = [&](int at, int j, float x) {
        kept[at] = j;
        if (at < new_width) out[at] = x;
    };
    // the candidates: this CTA's are `count` from key `base` on
    const int room = p.keep - p.sinks - p.recent;  // for fewer than all of them, where L > keep
    const bool choose = L > p.keep && room > 0;
    const int candidates = L - p.sinks - p.recent, each = (candidates + ctas - 1) / ctas;
    const int base = p.sinks + min(cta * each, candidates), count = min(each, p.sinks + candidates - base);
    const int held = min(count, p.cached);
    float v[kBatch];
    auto load = [&](int j0) {  // all of a thread's loads in flight
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int j = j0 + i * kThreads + tid;
            v[i] = j < held ? w[base + j] : 0.f;
        }
    };
    if (choose) {
        load(0);
        for (int i = tid; i < 3 * kBins; i += kThreads) hist[0][i] = 0;
    }
    if (bh % p.Hkv == 0 && all == 0) p.new_lens[b] = n;
    for (int i = n + all; i < p.keep; i += step) kept[i] = -1;
    for (int i = n + all; i < new_width; i += step) out[i] = 0.f;
    if (L <= p.keep) {
        for (int i = all; i < L; i += step) store(i, i, w[i]);
        return;
    }
    for (int i = all; i < p.sinks; i += step) store(i, i, w[i]);
    for (int i = all; i < p.recent; i += step) store(p.keep - p.recent + i, L - p.recent + i, w[L - p.recent + i]);
    if (!choose) return;
    for (int j0 = 0; j0 < held; j0 += kBatch * kThreads) {
        if (j0 > 0) load(j0);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int j = j0 + i * kThreads + tid;
            if (j < held) cached[j] = order(v[i]);
        }
    }
    __syncthreads();

    auto rank = [&](int j) { return j < held ? cached[j] : order(w[base + j]); };
    uint32_t last = 0, left = static_cast<uint32_t>(room);  // the rank of the last key that stays, so far; keys of it that stay
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        uint32_t *h = hist[pass];
#pragma unroll 4
        for (int j = tid; j < count; j += kThreads) {
            const uint32_t k = rank(j);
            if (pass == 0 || (k ^ last) >> (shift + bits) == 0) atomicAdd(&h[(k >> shift) & ((1u << bits) - 1)], 1u);
        }
        sync();
        // bins from the top, two a lane: a warp sums its own, over the cluster (all
        // of the other CTAs' counts are on their way at once)
        const int top = kBins - 2 - 2 * lane, here = top - warp * kOfWarp;  // the lower one of the two
        uint2 mine = *reinterpret_cast<const uint2 *>(h + here), other[kMaxCtas - 1];
#pragma unroll
        for (int x = 1; x < kMaxCtas; ++x) {
            const int rank = cta + x < ctas ? cta + x : cta + x - ctas;
            other[x - 1] = x < ctas ? *reinterpret_cast<const uint2 *>(cluster.map_shared_rank(h, static_cast<unsigned>(rank)) + here)
                                    : make_uint2(0u, 0u);
        }
#pragma unroll
        for (int x = 0; x < kMaxCtas - 1; ++x) {
            mine.x += other[x].x;
            mine.y += other[x].y;
        }
        *reinterpret_cast<uint2 *>(sum + here) = mine;
        const uint32_t own = __reduce_add_sync(kFull, mine.x + mine.y);
        if (lane == 0) of_warp[pass][warp] = own;
        __syncthreads();
        // the warp, the lane and the bin in which the count of keys from the top reaches `left`
        const uint32_t v = of_warp[pass][lane];
        uint32_t upto = scan(v);
        int at = __ffs(__ballot_sync(kFull, upto >= left)) - 1;
        left -= __shfl_sync(kFull, upto - v, at);
        const int low = top - at * kOfWarp;
        const uint2 two = *reinterpret_cast<const uint2 *>(sum + low);
        upto = scan(two.x + two.y);
        at = __ffs(__ballot_sync(kFull, upto >= left)) - 1;
        left -= __shfl_sync(kFull, upto - two.x - two.y, at);
        int bin = __shfl_sync(kFull, low, at);
        const uint32_t upper = __shfl_sync(kFull, two.y, at), lower = __shfl_sync(kFull, two.x, at);
        const bool in_upper = upper >= left;
        if (in_upper) ++bin;
        else left -= upper;
        last |= static_cast<uint32_t>(bin) << shift;
        // all keys with these digits stay (mostly so after two of them): no more to find
        if (left == (in_upper ? upper : lower) && last > 0) {
            --last;
            left = 0;
            break;
        }
    }
    // the keys above `last`, and the first `left` of its equals, in order
    const int run = (count + kWarps * 32 - 1) / (kWarps * 32) * 32;  // keys of a warp
    const int j0 = min(warp * run, count), j1 = min(j0 + run, count);
    auto load_run = [&](int i0) {  // (ahead of their stores)
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int j = i0 + 32 * i + lane;
            v[i] = j < j1 ? w[base + j] : 0.f;
        }
    };
    uint32_t up[kBatch], eq[kBatch];  // lanes whose key is above, equal
    auto compare = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int j = i0 + 32 * i + lane;
            up[i] = eq[i] = 0;
            if (j - lane >= j1) continue;
            const uint32_t k = j < j1 ? rank(j) : 0u;
            up[i] = __ballot_sync(kFull, j < j1 && k > last);
            eq[i] = __ballot_sync(kFull, j < j1 && k == last);
        }
    };
    load_run(j0);
    uint32_t above = 0, equal = 0;
    constexpr int kStep = 32 * kBatch;
    for (int i0 = j0 + max(j1 - j0 - 1, 0) / kStep * kStep; i0 >= j0; i0 -= kStep) {  // (the first ones last: they are needed next)
        compare(i0);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            above += __popc(up[i]);
            equal += __popc(eq[i]);
        }
    }
    if (lane == 0) counts[warp] = make_uint2(above, equal);
    sync();
    above = equal = 0;  // of the warps before this one
    for (int x = 0; x <= cta; ++x) {
        const uint2 *c = x == cta ? counts : cluster.map_shared_rank(counts, static_cast<unsigned>(x));
        if (lane < (x == cta ? warp : kWarps)) {
            const uint2 v = c[lane];
            above += v.x;
            equal += v.y;
        }
    }
    above = __reduce_add_sync(kFull, above);
    equal = __reduce_add_sync(kFull, equal);
    if (ctas > 1) cluster.barrier_arrive();  // (this CTA has read what it needs of the others)
    const unsigned before = (1u << lane) - 1;
    for (int i0 = j0; i0 < j1; i0 += kStep) {
        if (i0 > j0) {
            load_run(i0);
            compare(i0);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (i0 + 32 * i >= j1) break;
            const uint32_t a = above + __popc(up[i] & before), e = equal + __popc(eq[i] & before);
            if ((up[i] >> lane & 1) || ((eq[i] >> lane & 1) && e < left))
                store(p.sinks + static_cast<int>(a + min(e, left)), base + i0 + 32 * i + lane, v[i]);
            above += __popc(up[i]);
            equal += __popc(eq[i]);
        }
    }
    if (ctas > 1) cluster.barrier_wait();  // the others have read what they need of this one
}

constexpr int kCopyThreads = 128;
constexpr int kInFlight = 2;  // keys of a lane group with their loads in flight (4: 102 us becomes 108 where 16000 stay)

template <int D>
__global__ void __launch_bounds__(kCopyThreads) fa_kv_evict_copy_kernel(const EvictParams p) {
    constexpr int kLanes = D / 8, kGroups = kCopyThreads / kLanes;
    const long long bh = static_cast<long long>(blockIdx.z) * gridDim.y + blockIdx.y;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    if (bh >= static_cast<long long>(p.B) * p.Hkv) return;
    const int b = static_cast<int>(bh / p.Hkv), hk = static_cast<int>(bh % p.Hkv);
    const int n = min(min(max(p.seq_lens[b], 0), p.max_blocks << p.log2_bs), p.keep);
    const int r0 = static_cast<int>(blockIdx.x) * kGroups * kInFlight + static_cast<int>(threadIdx.x) / kLanes;
    const int col = static_cast<int>(threadIdx.x) % kLanes * 8, mask = (1 << p.log2_bs) - 1;
    if (static_cast<int>(blockIdx.x) * kGroups * kInFlight >= n) return;
    uint4 k[kInFlight], v[kInFlight];
    long long dst[kInFlight];
    int j[kInFlight];
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
        const int r = r0 + i * kGroups;
        j[i] = r < n ? __ldcg(p.kept + bh * p.keep + r) : -1;
    }
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
        const int r = r0 + i * kGroups;
        dst[i] = -1;
        if (r >= n) continue;
        const int from = p.block_table[static_cast<size_t>(b) * p.max_blocks + (j[i] >> p.log2_bs)];
        const int to = (r >> p.log2_bs) < p.new_max_blocks
                           ? p.new_table[static_cast<size_t>(b) * p.new_max_blocks + (r >> p.log2_bs)]
                           : -1;
        if (static_cast<unsigned>(from) >= static_cast<unsigned>(p.num_blocks) ||
            static_cast<unsigned>(to) >= static_cast<unsigned>(p.num_blocks)) {
            atomicExch(p.err, kDeviceErrBadIndex);
            continue;
        }
        const long long src = ((((static_cast<long long>(from) * p.Hkv + hk) << p.log2_bs) + (j[i] & mask)) * D) + col;
        dst[i] = ((((static_cast<long long>(to) * p.Hkv + hk) << p.log2_bs) + (r & mask)) * D) + col;
        k[i] = __ldcs(reinterpret_cast<const uint4 *>(p.k_cache + src));
        v[i] = __ldcs(reinterpret_cast<const uint4 *>(p.v_cache + src));
    }
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
        if (dst[i] < 0) continue;
        *reinterpret_cast<uint4 *>(p.k_cache + dst[i]) = k[i];
        *reinterpret_cast<uint4 *>(p.v_cache + dst[i]) = v[i];
    }
}

}  // namespace evict

cudaError_t launch_kv_evict(int D, EvictParams p, int sms, cudaStream_t st) {
    static std::atomic<unsigned long long> done{0};
    const long long width = static_cast<long long>(p.max_blocks) << p.log2_bs;
    const unsigned units = static_cast<unsigned>(p.B) * static_cast<unsigned>(p.Hkv);
    // a cluster of as many CTAs as there are SMs and keys (a thousand each) for
    int ctas = 1;
    while (ctas < evict::kMaxCtas && 2LL * ctas * units <= sms && width > 1024LL * ctas) ctas *= 2;
    const long long each = (width + ctas - 1) / ctas;
    p.cached = static_cast<int>(each < evict::kMaxCached ? each : evict::kMaxCached);
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(evict::fa_kv_evict_select_kernel),
                               evict::kMaxCached * static_cast<int>(sizeof(uint32_t)), done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeClusterDimension;
    attrs[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attrs[0].val.clusterDim.y = 1;
    attrs[0].val.clusterDim.z = 1;
    attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // as launch_early
    attrs[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t sel = {};
    sel.gridDim = dim3(units * static_cast<unsigned>(ctas));
    sel.blockDim = dim3(evict::kThreads);
    sel.dynamicSmemBytes = static_cast<size_t>(p.cached) * sizeof(uint32_t);
    sel.stream = st;
    sel.attrs = attrs;
    sel.numAttrs = 2;
    e = cudaLaunchKernelEx(&sel, evict::fa_kv_evict_select_kernel, p);
    if (e != cudaSuccess) return e;
    const unsigned rows = static_cast<unsigned>(evict::kCopyThreads / (D / 8) * evict::kInFlight);
    const unsigned long long most = width < p.keep ? static_cast<unsigned long long>(width) : p.keep;
    const unsigned y = units < 65535u ? units : 65535u;
    const dim3 grid(static_cast<unsigned>((most + rows - 1) / rows), y, (units + y - 1) / y);
    return launch_early(D == 64 ? evict::fa_kv_evict_copy_kernel<64> : evict::fa_kv_evict_copy_kernel<128>, grid,
                        evict::kCopyThreads, 0, st, true, p);
}

}  // namespace fa
