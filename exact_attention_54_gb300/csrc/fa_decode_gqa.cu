// One-token attention over a paged cache whose key heads are shared by groups
// of query heads, with a sliding window and sinks: 16-bit pages
// (fa_decode_paged_window) or the 4-bit cache (fa_decode_paged_q4).
//
// Split-KV as in fa_decode.cu: partial (m, l, O) per partition of the visible
// keys, the last partition of a key head to finish merges its query heads.
// Visible index i of a sequence of L keys is key i for i < n_sink, and key
// i + skip after that, with n_sink = min(sinks, L - window) (no sinks apart
// from the window where the window reaches them) and skip the hidden stretch.
#include <math_constants.h>

#include "fa_kv_q4.cuh"
#include "fa_launch.h"

namespace fa {
namespace gqa {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kHeads = 8;  // query heads per pass over the keys

// grid: (b * Hkv + key head) * num_splits + partition
template <int D, bool BF16, bool Q4>
__global__ void __launch_bounds__(kThreads) fa_decode_gqa_kernel(const GqaDecodeParams p) {
    constexpr int E = D / 32;  // columns per lane: lane + 32 e
    __shared__ float sm_m[kWarps][kHeads], sm_l[kWarps][kHeads], sm_o[kWarps][kHeads][D];
    const int S = p.num_splits;
    const int s = static_cast<int>(blockIdx.x) % S, bk = static_cast<int>(blockIdx.x) / S;
    const int b = bk / p.Hkv, hk = bk % p.Hkv;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int cap = p.max_blocks << p.log2_bs;
    const int L = min(max(p.seq_lens[b], 0), cap);
    const int w_lo = p.window > 0 ? max(L - p.window, 0) : 0;
    const int n_sink = min(p.sinks, w_lo);
    const int n_vis = n_sink + L - w_lo, skip = w_lo - n_sink;
    const int part = (n_vis + S - 1) / S;
    const int lo = min(s * static_cast<long long>(part), static_cast<long long>(n_vis));
    const int hi = min(lo + part, n_vis);
    const int *table = p.block_table + static_cast<size_t>(b) * p.max_blocks;
    bool bad_page = false;

    for (int g0 = 0; g0 < p.group; g0 += kHeads) {
        const int heads = min(kHeads, p.group - g0);
        const size_t bh0 = static_cast<size_t>(b) * p.H + hk * p.group + g0;
        float m[kHeads], l[kHeads], acc[kHeads][E];
        for (int h = 0; h < kHeads; ++h) {
            m[h] = -CUDART_INF_F;
            l[h] = 0.f;
            for (int e = 0; e < E; ++e) acc[h][e] = 0.f;
        }
        for (int i = lo + warp; i < hi; i += kWarps) {
            const int key = i < n_sink ? i : i + skip;
            const int page = table[key >> p.log2_bs];
            if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_blocks)) {
                bad_page = true;
                continue;
            }
            const size_t row = ((static_cast<size_t>(page) * p.Hkv + hk) << p.log2_bs) + (key & ((1 << p.log2_bs) - 1));
            float kv[E], vv[E];
            for (int e = 0; e < E; ++e) {
                const int d = lane + 32 * e;
                if constexpr (Q4) {
                    const size_t at = row * (D / 2) + q4::code_byte<D>(d);
                    const int kc = (static_cast<const uint8_t *>(p.k)[at] >> (4 * (d % 2))) & 15;
                    const int vc = (static_cast<const uint8_t *>(p.v)[at] >> (4 * (d % 2))) & 15;
                    const size_t sat = row * (D / q4::kGroup) + e;
                    kv[e] = static_cast<float>(kc - 8) * q4::from16<BF16>(static_cast<const uint16_t *>(p.ks)[sat]);
                    vv[e] = static_cast<float>(vc - 8) * q4::from16<BF16>(static_cast<const uint16_t *>(p.vs)[sat]);
                } else {
                    kv[e] = q4::from16<BF16>(static_cast<const uint16_t *>(p.k)[row * D + d]);
                    vv[e] = q4::from16<BF16>(static_cast<const uint16_t *>(p.v)[row * D + d]);
                }
            }
            for (int h = 0; h < kHeads; ++h) {
                if (h >= heads) break;
                float x = 0.f;
                for (int e = 0; e < E; ++e) x = fmaf(q4::from16<BF16>(p.q[(bh0 + h) * D + lane + 32 * e]), kv[e], x);
                for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
                x *= p.scale_log2;
                const float m_new = fmaxf(m[h], x);
                const float a = m_new == -CUDART_INF_F ? 1.f : ptx::ex2(m[h] - m_new), w = ptx::ex2(x - m_new);
                l[h] = l[h] * a + w;
                for (int e = 0; e < E; ++e) acc[h][e] = acc[h][e] * a + w * vv[e];
                m[h] = m_new;
            }
        }
        __syncthreads();
        for (int h = 0; h < kHeads; ++h) {
            if (lane == 0) {
                sm_m[warp][h] = m[h];
                sm_l[warp][h] = l[h];
            }
            for (int e = 0; e < E; ++e) sm_o[warp][h][lane + 32 * e] = acc[h][e];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < heads * D; i += kThreads) {
            const int h = i / D, d = i % D;
            float M = -CUDART_INF_F, Lw = 0.f, O = 0.f;
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w][h]);
            for (int w = 0; w < kWarps; ++w) {
                const float f = M == -CUDART_INF_F ? 1.f : ptx::ex2(sm_m[w][h] - M);
                Lw = fmaf(f, sm_l[w][h], Lw);
                O = fmaf(f, sm_o[w][h][d], O);
            }
            const size_t at = (bh0 + h) * S + s;
            p.o_part[at * D + d] = O;
            if (d == 0) {
                p.m_part[at] = M;
                p.l_part[at] = Lw;
            }
        }
    }
    if (bad_page) atomicExch(p.err, kDeviceErrBadIndex);

    // the last partition of this key head merges its query heads
    __shared__ int is_last;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) is_last = atomicAdd(p.counters + bk, 1) == S - 1;
    __syncthreads();
    if (!is_last) return;
    __threadfence();
    for (int i = threadIdx.x; i < p.group * D; i += kThreads) {
        const size_t bh = static_cast<size_t>(b) * p.H + hk * p.group + i / D;
        const int d = i % D;
        float M = -CUDART_INF_F, Lw = 0.f, O = 0.f;
        for (int j = 0; j < S; ++j) M = fmaxf(M, __ldcg(p.m_part + bh * S + j));
        for (int j = 0; j < S; ++j) {
            const float f = M == -CUDART_INF_F ? 1.f : ptx::ex2(__ldcg(p.m_part + bh * S + j) - M);
            Lw = fmaf(f, __ldcg(p.l_part + bh * S + j), Lw);
            O = fmaf(f, __ldcg(p.o_part + (bh * S + j) * D + d), O);
        }
        // no visible key: O = 0 and LSE = -inf; a NaN stays one
        static_cast<uint16_t *>(p.o)[bh * D + d] = q4::to16<BF16>(Lw == 0.f ? 0.f : O / Lw);
        if (d == 0) p.lse[bh] = Lw == 0.f ? -CUDART_INF_F : (M + log2f(Lw)) * 0.69314718055994531f;
    }
    if (threadIdx.x == 0) p.counters[bk] = 0;
}

template <int D, bool BF16>
static cudaError_t launch_t(bool q4, const GqaDecodeParams &p, unsigned grid, cudaStream_t st) {
    if (q4) fa_decode_gqa_kernel<D, BF16, true><<<grid, kThreads, 0, st>>>(p);
    else fa_decode_gqa_kernel<D, BF16, false><<<grid, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace gqa

int decode_gqa_splits(int sms, int B, int, int Hkv, int max_keys) {
    const long long heads = static_cast<long long>(B) * Hkv;
    long long s = (4LL * sms + heads - 1) / heads;  // four CTAs per SM
    const long long most = (max_keys + 63) / 64;    // at least 64 keys each
    s = s < most ? s : most;
    return static_cast<int>(s < 64 ? s : 64);
}

cudaError_t launch_decode_gqa(int D, bool bf16, bool q4, const GqaDecodeParams &p, int grid, cudaStream_t st) {
    const unsigned g = static_cast<unsigned>(grid);
    if (D == 64) return bf16 ? gqa::launch_t<64, true>(q4, p, g, st) : gqa::launch_t<64, false>(q4, p, g, st);
    return bf16 ? gqa::launch_t<128, true>(q4, p, g, st) : gqa::launch_t<128, false>(q4, p, g, st);
}

}  // namespace fa
