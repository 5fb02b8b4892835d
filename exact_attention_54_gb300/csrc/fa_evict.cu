// Eviction from a paged 16-bit cache by accumulated attention weight
// (fa_kv_evict): of each sequence and key head the first `sinks` keys, the last
// `recent` and the heaviest between them stay, in their order, in new pages.
//
// Two launches. Selection: a cluster of CTAs per (sequence, key head), as many as
// there are SMs for, each with a run of its keys, finds the weight of the last key
// that stays as an order statistic, digit by digit from the top (11, 11 and 10
// bits of the weight's bits, ordered as integers; the CTAs add up their counts
// through distributed shared memory), then writes the keys above it, and as many of
// the equal ones as there is room for, by prefix sums over the keys. The weights
// are read from memory once and kept in shared memory, as far as they fit. Copy:
// lane groups of 16-byte pieces, page by table on both sides; a stream of 2 D bytes
// read and written per key and value.
//
// Bound: the copy by HBM; the selection by instruction issue.
#include <cooperative_groups.h>

#include "fa_launch.h"
#include "sm103_ptx.cuh"

namespace fa {
namespace evict {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCached = 46 * 1024;  // keys whose weights shared memory holds
constexpr int kBins = 2048;
constexpr int kEach = 4;               // consecutive keys of a thread, compaction
constexpr unsigned kFull = 0xffffffffu;

// A weight's bits, ordered like the weights as unsigned integers: -0 is +0, a NaN is below everything.
__device__ __forceinline__ uint32_t order(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// Sum of v over the threads before this one; `total`: over all. The whole CTA calls it.
__device__ __forceinline__ uint32_t prefix_sum(uint32_t v, uint32_t *sums, uint32_t &total) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint32_t x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(kFull, x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();  // sums of the previous call are read
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        uint32_t s = sums[lane];
#pragma unroll
        for (int off = 1; off < kWarps; off <<= 1) {
            const uint32_t y = __shfl_up_sync(kFull, s, off);
            if (lane >= off) s += y;
        }
        sums[lane] = s;
    }
    __syncthreads();
    total = sums[kWarps - 1];
    return x - v + (warp > 0 ? sums[warp - 1] : 0u);
}

__global__ void __launch_bounds__(kThreads, 1) fa_kv_evict_select_kernel(const EvictParams p) {
    extern __shared__ uint4 cached4[];  // the order of this CTA's first p.cached keys
    __shared__ uint32_t hist[3][kBins], sums[kWarps], pick[2], mine[2];
    uint32_t *cached = reinterpret_cast<uint32_t *>(cached4);
    auto cluster = cooperative_groups::this_cluster();
    const int ctas = static_cast<int>(cluster.num_blocks()), cta = static_cast<int>(cluster.block_rank());
    const int tid = static_cast<int>(threadIdx.x), all = cta * kThreads + tid, step = ctas * kThreads;
    ptx::grid_launch_dependents();
    const size_t bh = blockIdx.x / ctas;
    const int b = static_cast<int>(bh / p.Hkv);
    const int width = p.max_blocks << p.log2_bs, new_width = p.new_max_blocks << p.log2_bs;
    const int L = min(max(p.seq_lens[b], 0), width), n = min(L, p.keep);
    const float *w = p.weights + bh * width;
    int *kept = p.kept + bh * p.keep;
    float *out = p.new_weights + bh * new_width;
    auto store = [&](int at, int j) {
        kept[at] = j;
        if (at < new_width) out[at] = w[j];
    };
    if (bh % p.Hkv == 0 && all == 0) p.new_lens[b] = n;
    for (int i = n + all; i < p.keep; i += step) kept[i] = -1;
    for (int i = n + all; i < new_width; i += step) out[i] = 0.f;
    if (L <= p.keep) {
        for (int i = all; i < L; i += step) store(i, i);
        return;
    }
    for (int i = all; i < p.sinks; i += step) store(i, i);
    for (int i = all; i < p.recent; i += step) store(p.keep - p.recent + i, L - p.recent + i);
    const int room = p.keep - p.sinks - p.recent;  // fewer than the candidates
    if (room == 0) return;

    // this CTA's candidates: count of them from key `base` on
    const int candidates = L - p.sinks - p.recent, each = (candidates + ctas - 1) / ctas;
    const int base = p.sinks + min(cta * each, candidates), count = min(each, p.sinks + candidates - base);
    const int held = min(count, p.cached);
    for (int j0 = 0; j0 < held; j0 += 8 * kThreads) {  // eight loads of a thread in flight
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = j0 + i * kThreads + tid;
            x[i] = j < held ? w[base + j] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = j0 + i * kThreads + tid;
            if (j < held) cached[j] = order(x[i]);
        }
    }
    for (int i = tid; i < 3 * kBins; i += kThreads) hist[0][i] = 0;
    __syncthreads();
    // the orders of candidates j .. j + 3 (0 behind the last)
    auto four = [&](int j, uint32_t (&k)[kEach]) {
        if (j + kEach <= held) {
            const uint4 v = cached4[j / kEach];
            k[0] = v.x;
            k[1] = v.y;
            k[2] = v.z;
            k[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                k[i] = j + i < held ? cached[j + i] : j + i < count ? order(w[base + j + i]) : 0u;
        }
    };
    uint32_t last = 0, left = static_cast<uint32_t>(room);  // the rank of the last key that stays, so far; keys of it that stay
    uint32_t above = 0;                                     // of this CTA's keys, in this thread's bins
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        uint32_t *h = hist[pass];
        for (int j = tid * kEach; j < count; j += kThreads * kEach) {
            uint32_t k[kEach];
            four(j, k);
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (j + i < count && (pass == 0 || (k[i] ^ last) >> (shift + bits) == 0))
                    atomicAdd(&h[(k[i] >> shift) & ((1u << bits) - 1)], 1u);
        }
        cluster.sync();
        // bins from the top, two a thread: the one in which the count of keys reaches `left`
        const int top = kBins - 1 - 2 * tid;
        const uint32_t l0 = h[top], l1 = h[top - 1];
        uint32_t c0 = l0, c1 = l1;
        for (int c = 1; c < ctas; ++c) {
            const uint32_t *other = cluster.map_shared_rank(h, static_cast<unsigned>((cta + c) % ctas));
            c0 += other[top];
            c1 += other[top - 1];
        }
        uint32_t total;
        const uint32_t before = prefix_sum(c0 + c1, sums, total);
        if (before < left && left <= before + c0 + c1) {
            const bool first = left <= before + c0;
            pick[0] = static_cast<uint32_t>(first ? top : top - 1);
            pick[1] = left - (first ? before : before + c0);
        }
        __syncthreads();
        const int bin = static_cast<int>(pick[0]);
        above += (top > bin ? l0 : 0u) + (top - 1 > bin ? l1 : 0u);
        last |= static_cast<uint32_t>(bin) << shift;
        left = pick[1];
    }
    // keys above `last`, and its equals, of the CTAs before this one
    uint32_t at_above = 0, at_equal = 0;
    {
        uint32_t total;
        prefix_sum(above, sums, total);
        if (tid == 0) {
            mine[0] = total;
            mine[1] = hist[2][last & 1023u];
        }
        cluster.sync();
        for (int c = 0; c < cta; ++c) {
            const uint32_t *other = cluster.map_shared_rank(mine, static_cast<unsigned>(c));
            at_above += other[0];
            at_equal += other[1];
        }
    }
    // the keys above `last`, and the first `left` of its equals, in order
    for (int j0 = 0; j0 < count; j0 += kThreads * kEach) {
        const int j = j0 + tid * kEach;
        uint32_t k[kEach], some = 0;  // above: upper 16 bits, equal: lower
        four(j, k);
#pragma unroll
        for (int i = 0; i < kEach; ++i) some += j + i >= count ? 0u : k[i] > last ? 0x10000u : k[i] == last ? 1u : 0u;
        uint32_t total;
        const uint32_t before = prefix_sum(some, sums, total);
        uint32_t a = at_above + (before >> 16), e = at_equal + (before & 0xffffu);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (j + i >= count) break;
            if (k[i] > last) {
                store(p.sinks + static_cast<int>(a + min(e, left)), base + j + i);
                ++a;
            } else if (k[i] == last) {
                if (e < left) store(p.sinks + static_cast<int>(a + e), base + j + i);
                ++e;
            }
        }
        at_above += total >> 16;
        at_equal += total & 0xffffu;
    }
    cluster.sync();  // the others have read what they need of this CTA
}

constexpr int kCopyThreads = 128;
constexpr int kInFlight = 4;  // keys of a lane group with their loads in flight

template <int D>
__global__ void __launch_bounds__(kCopyThreads) fa_kv_evict_copy_kernel(const EvictParams p) {
    constexpr int kLanes = D / 8, kGroups = kCopyThreads / kLanes;
    const long long bh = static_cast<long long>(blockIdx.z) * gridDim.y + blockIdx.y;
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
    // a cluster of up to 8 CTAs (the portable size) where SMs and keys (a thousand each) are there for them
    int ctas = 1;
    while (ctas < 8 && 2LL * ctas * units <= sms && width > 1024LL * ctas) ctas *= 2;
    const long long each = (width + ctas - 1) / ctas;
    p.cached = static_cast<int>(each < evict::kMaxCached ? (each + 3) / 4 * 4 : evict::kMaxCached);
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(evict::fa_kv_evict_select_kernel),
                               evict::kMaxCached * static_cast<int>(sizeof(uint32_t)), done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute cluster[1];
    cluster[0].id = cudaLaunchAttributeClusterDimension;
    cluster[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    cluster[0].val.clusterDim.y = 1;
    cluster[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t sel = {};
    sel.gridDim = dim3(units * static_cast<unsigned>(ctas));
    sel.blockDim = dim3(evict::kThreads);
    sel.dynamicSmemBytes = static_cast<size_t>(p.cached) * sizeof(uint32_t);
    sel.stream = st;
    sel.attrs = cluster;
    sel.numAttrs = 1;
    e = cudaLaunchKernelEx(&sel, evict::fa_kv_evict_select_kernel, p);
    if (e != cudaSuccess) return e;
    const unsigned rows = static_cast<unsigned>(evict::kCopyThreads / (D / 8) * evict::kInFlight);
    const unsigned long long most = width < p.keep ? static_cast<unsigned long long>(width) : p.keep;
    const unsigned y = units < 65535u ? units : 65535u;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((most + rows - 1) / rows), y, (units + y - 1) / y);
    cfg.blockDim = dim3(evict::kCopyThreads);
    cfg.stream = st;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return D == 64 ? cudaLaunchKernelEx(&cfg, evict::fa_kv_evict_copy_kernel<64>, p)
                   : cudaLaunchKernelEx(&cfg, evict::fa_kv_evict_copy_kernel<128>, p);
}

}  // namespace fa
