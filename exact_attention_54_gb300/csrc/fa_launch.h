// Internal interface between the C ABI (fa_api.cu) and the kernel translation
// units. Not installed, not part of the public header.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

namespace fa {

// Lets a kernel use `bytes` of dynamic shared memory on the current device.
// Set once per device and kernel (`done`: a static of the caller's, one bit
// per device): the attribute stays, and setting it costs a launch's time.
inline cudaError_t allow_smem(const void *kern, int bytes, std::atomic<unsigned long long> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Values written to the device error word: a kernel abandoned a wait, met an
// out-of-range device-side index (a page number in a block table), or found
// packed-sequence offsets that do not describe sequences inside the tensors
// (or a query sequence longer than the launch was sized for).
constexpr int kDeviceErrTimeout = 1;
constexpr int kDeviceErrBadIndex = 2;
constexpr int kDeviceErrSeqLens = 3;

// Default bound on any single wait on an on-chip barrier.
constexpr unsigned long long kWaitTimeoutNs = 1000000000ull;  // 1 s

// Parameters of the forward kernel (dense and packed-varlen layouts).
struct FwdParams {
    void *o;               // [B,H,Sq,D] dense | [total_q,H,D] varlen
    float *lse;            // [B,H,Sq]   dense | [H,total_q]   varlen
    const int *cu_q;       // varlen only: int32[B+1]
    const int *cu_k;       // varlen only: int32[B+1]
    int B;                 // batch size (dense) or number of sequences (varlen)
    int H;                 // heads
    int Sq;                // query length (dense) or max query length (varlen)
    int Sk;                // key length (dense only)
    int total_q;           // varlen: LSE row stride of one head
    int total_k;           // varlen: key tokens (bound of cu_k)
    int n_pairs;           // query-tile pairs per (sequence, head): ceil(ceil(Sq/128)/2)
    int n_qtiles;          // 128-row query tiles per (sequence, head): ceil(Sq/128)
    int num_work;          // work items: n_pairs * B * H (D <= 128), n_qtiles * B * H * D / 256 (D >= 256)
    float scale_log2;      // scale * log2(e)
    int *err;              // device error word
    unsigned long long timeout_ns;
    int withhold;          // test support, 0 = off: CTA 0 never issues its V tile load number withhold - 1
    int window, sinks;     // sliding window only: keys a query sees back to itself; first keys always visible
    int group;             // sliding window only: query heads per key head
};

int fwd_smem_bytes(int D);

// A packed sequence whose offsets [q0, q1) and [k0, k1) do not lie inside the
// tensors (0 <= begin <= end <= total), or whose query length exceeds p.Sq
// (the max_seqlen_q the launch was sized for).
__device__ __forceinline__ bool varlen_seq_bad(const FwdParams &p, int q0, int q1, int k0, int k1) {
    return q0 < 0 || q1 < q0 || q1 > p.total_q || q1 - q0 > p.Sq || k0 < 0 || k1 < k0 || k1 > p.total_k;
}

// Packed-sequence offsets check, run by every thread of a CTA (all must call
// it): true when no sequence is bad. Every CTA reaches the same answer;
// thread 0 of each CTA that finds a fault records it in the device error word.
__device__ __forceinline__ bool varlen_offsets_ok(const FwdParams &p) {
    bool bad = false;
    for (int b = static_cast<int>(threadIdx.x); b < p.B; b += static_cast<int>(blockDim.x))
        bad |= varlen_seq_bad(p, p.cu_q[b], p.cu_q[b + 1], p.cu_k[b], p.cu_k[b + 1]);
    bad = __syncthreads_or(bad) != 0;
    if (bad && threadIdx.x == 0) atomicExch(p.err, kDeviceErrSeqLens);
    return !bad;
}

// Parameters of the split-KV decode kernel (dense and paged K/V).
struct DecodeParams {
    const uint16_t *q, *k, *v;   // q [B*H, D]; k, v dense [B*H, Sk, D] or pages [num_blocks, H, bs, D]
    float *o_part, *m_part, *l_part;
    int H;                       // heads (paged: to locate the head inside a page)
    int Sk;                      // dense: keys per head
    int num_splits;
    int keys_per_split;          // dense: ceil(Sk / num_splits)
    float scale_log2;
    const int *block_table;      // paged: [B, max_blocks] page numbers
    const int *seq_lens;         // paged: [B] keys per sequence
    int max_blocks;              // paged: row length of block_table
    int log2_bs;                 // paged: log2(block_size)
    int num_blocks;              // paged: pages in the cache
    int *err;                    // paged: device error word
    void *o;                     // fused: [B*H, D] output (input dtype)
    float *lse;                  // fused: [B*H] log-sum-exp
    int *counters;               // fused: [B*H] finished partitions per head, zero between calls
};

// Parameters of the backward pass: dense [B,H,S,D] or packed [T,H,D] layout.
// A work unit is a head (dense) or a (sequence, head) pair (packed).
struct BwdParams {
    float *lse2;           // dense [B*H][Sq_pad], +inf past Sq | packed [H][total_q]: forward LSE * log2(e)
    float *delta;          // same layout: D_i = sum_d dO_id O_id (0 past Sq, dense)
    float *dq_acc;         // dense [B*H][Sq][D] | packed [total_q][H][D]: fp32 accumulator of dS K
    void *dk, *dv;         // dense [B*H][Sk][D] | packed [total_k][H][D] outputs (input dtype)
    int BH;                // work units: B*H (dense), num_seqs*H (packed)
    int Sq, Sk;            // dense: lengths; packed: max_seqlen_q, max_seqlen_k
    int Sq_pad;            // dense: Sq rounded up to whole 128-row tiles
    int n_qtiles, n_ktiles;
    int heads_per_group;   // CTAs run work units group by group (see bwd_work)
    const int *cu_q;       // packed: int32[num_seqs + 1]
    const int *cu_k;       // packed: int32[num_seqs + 1]
    int H;                 // packed: heads
    int total_q, total_k;  // packed: tokens
    float scale, scale_log2;
    int *err;              // device error word
    unsigned long long timeout_ns;
    int withhold;          // test support, 0 = off: the CTA with the first unit never issues its Q/dO load number withhold - 1
    int *work_counter;     // D = 128: next work unit to hand out (in the workspace, zeroed by the prep kernel)
    int total_units;       // D = 128: work units of the launch (BH * n_ktiles)
    int grid;              // D = 128: persistent CTAs (at most one per SM)
    int window, sinks;     // sliding window only: keys a query sees back to itself; first keys always visible
    int group;             // sliding window only: query heads per key head
    int units;             // sliding window only: key heads (dense B*Hkv, packed num_seqs*Hkv) that key tiles belong to
    int sink_tiles;        // sliding window only: key tiles that hold sinks (at most n_ktiles)
    int segs_sink, segs;   // sliding window only: segments of their steps, and of the other key tiles'
    float *segments;       // sliding window only: the segments' dV and dK (unused where both counts are 1)
};

// Test support: a launch that withholds one load (see FwdParams::withhold)
// leaves a wait that nothing completes, so the kernel's bounded wait runs
// out and its abort path (drain, TMEM release, error word) runs.
// `first`: whether this CTA has the launch's first work item (CTA 0, where
// items are handed out in block order).
__device__ __forceinline__ bool withheld(int withhold, uint32_t load, bool first) {
    return withhold > 0 && first && load + 1 == static_cast<uint32_t>(withhold);
}
__device__ __forceinline__ bool withheld(int withhold, uint32_t load) {
    return withheld(withhold, load, blockIdx.x == 0);
}

// maps: {Q, K, V, dO, dQ accumulator (fp32)}; lse dense [B*H][Sq] | packed
// [H][total_q]; dq output (input dtype). Dense maps are 3-D {D, S, B*H},
// packed maps {D, H, tokens}.
cudaError_t launch_bwd_dense(int D, bool bf16, bool causal, const CUtensorMap *maps, const void *o,
                             const void *dout, const float *lse, void *dq, const BwdParams &p, cudaStream_t stream);
cudaError_t launch_bwd_varlen(int D, bool bf16, bool causal, const CUtensorMap *maps, const void *o,
                              const void *dout, const float *lse, void *dq, const BwdParams &p, cudaStream_t stream);

// Sliding window and sinks, shared key heads: maps as above, K and V maps over
// H / p.group heads; p.BH and p.H count query heads.
cudaError_t launch_bwd_window(int D, bool bf16, bool varlen, const CUtensorMap *maps, const void *o,
                              const void *dout, const float *lse, void *dq, const BwdParams &p, cudaStream_t stream);

// maps: {Q, K, V} tensor maps (see fa_api.cu for their geometry).
cudaError_t launch_fwd_dense(int D, bool bf16, bool causal, const CUtensorMap *maps,
                             const FwdParams &p, int grid, cudaStream_t stream);
cudaError_t launch_fwd_varlen(int D, bool bf16, bool causal, const CUtensorMap *maps,
                              const FwdParams &p, int grid, cudaStream_t stream);
// Sliding window and sinks, shared key heads (D = 64, 128): maps as above, K
// and V maps over H / p.group heads.
cudaError_t launch_fwd_window(int D, bool bf16, bool varlen, const CUtensorMap *maps, const FwdParams &p, int grid,
                              cudaStream_t stream);
// D = 256: one query tile per work item; maps: Q boxes of 128 rows, K/V boxes of 64.
cudaError_t launch_fwd_d256(bool bf16, bool causal, bool varlen, const CUtensorMap *maps, const FwdParams &p,
                            int grid, cudaStream_t stream);
// D = 512, 1024 (Split-D): one query tile and one 256-column output slice per
// work item; same maps (boxes of 64 columns; 128 rows for Q, 64 for K/V).
cudaError_t launch_fwd_splitd(int D, bool bf16, bool causal, bool varlen, const CUtensorMap *maps,
                              const FwdParams &p, int grid, cudaStream_t stream);

cudaError_t launch_decode_split(int D, bool bf16, const void *q, const void *k, const void *v,
                                float *o_part, float *m_part, float *l_part, int BH, int Sk,
                                int num_splits, int keys_per_split, float scale_log2,
                                cudaStream_t stream);

cudaError_t launch_decode_split_paged(int D, bool bf16, const DecodeParams &p, int BH, cudaStream_t stream);

// Phase 1 and phase 2 in one launch: the last partition of each head to
// finish merges that head (p.o, p.lse, p.counters must be set).
cudaError_t launch_decode_fused(int D, bool bf16, bool paged, const DecodeParams &p, int BH, cudaStream_t stream);

cudaError_t launch_splitkv_merge(int D, bool bf16, const float *o_part, const float *m_part,
                                 const float *l_part, void *o, float *lse, int BH,
                                 int num_splits, cudaStream_t stream);

// Parameters of the 4-bit cache's write and read kernels.
struct KvQ4Params {
    void *k, *v;                // packed rows [total, Hkv, D] (write: input, read: output)
    void *k_codes, *k_scales;   // pages [num_blocks, Hkv, block_size, D/2 and D/32]
    void *v_codes, *v_scales;
    const int *block_table;     // [num_seqs, max_blocks]
    const int *cu_seqlens;      // [num_seqs + 1]
    const int *starts;          // [num_seqs] or nullptr
    int total, max_seqlen, Hkv;
    int num_blocks, log2_bs, max_blocks;
    // set by kv_q4_grid: sequences, tokens per CTA, CTAs per sequence, and what
    // spares the kernels divisions by Hkv
    int num_seqs, tokens, chunks;
    unsigned inv_hkv;
    int step_t, step_h;
    int *err;                   // device error word
};

// CTAs of the write or read launch (sets the launch's fields of p).
long long kv_q4_grid(int D, int num_seqs, KvQ4Params &p);
cudaError_t launch_kv_q4(int D, bool bf16, bool write, const KvQ4Params &p, cudaStream_t stream);

// Parameters of the paged decode kernels with shared key heads.
struct GqaDecodeParams {
    const uint16_t *q;          // [B, H, D]
    const void *k, *v;          // pages: 16-bit rows, or code rows (4-bit)
    const void *ks, *vs;        // 4-bit: scale rows
    float *o_part, *m_part, *l_part;  // [B, H, num_splits(, D)]
    void *o;                    // [B, H, D]
    float *lse;                 // [B, H]
    int *counters;              // [B * H], one per key head and head tile: zero between calls
    const int *block_table;     // [B, max_blocks]
    const int *seq_lens;        // [B]
    int B, H, Hkv, group;       // sequences, query heads, key heads, H / Hkv
    bool balanced;              // the plan (set by decode_gqa_grid)
    int num_splits;
    int window, sinks;          // window 0: every key is visible
    int max_blocks, log2_bs, num_blocks;
    float scale_log2;
    int *err;                   // device error word
};

cudaError_t launch_decode_window(int D, bool bf16, const GqaDecodeParams &p, int sms, cudaStream_t stream);
cudaError_t launch_decode_q4(int D, bool bf16, const GqaDecodeParams &p, int sms, cudaStream_t stream);
// CTAs of either launch: a wave of ctas_per_sm per SM where the balanced plan
// serves, else one per unit (heads_per_unit query heads) and partition (sets p.balanced).
unsigned decode_gqa_grid(GqaDecodeParams &p, int sms, int ctas_per_sm, int heads_per_unit);
// Partitions that fill `sms` SMs (fa_decode_splits).
int decode_gqa_splits(int sms, int B, int H, int Hkv, int max_keys);

}  // namespace fa
