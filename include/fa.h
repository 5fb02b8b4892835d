/*
 * fa.h - C ABI of the GB300 (sm_103a) exact-attention library (libfa.so).
 *
 * Operations
 *   fa_fwd             FlashAttention-2 forward over dense [B,H,S,D] tensors.
 *   fa_fwd_varlen      the same forward over packed variable-length sequences.
 *   fa_decode_splitkv  split-KV decoding, phase 1: per-partition partials.
 *   fa_splitkv_merge   split-KV decoding, phase 2: log-sum-exp merge.
 *   fa_decode_splitkv_fused, fa_decode_paged_splitkv_fused
 *                      both phases in one launch (last partition merges).
 *   fa_bwd             backward pass: dQ, dK, dV from dO and the forward LSE.
 *   fa_fwd_window, fa_bwd_window (and _varlen)
 *                      forward and backward with a sliding window, sinks and
 *                      shared key heads.
 *   fa_kv_write_q4, fa_kv_read_q4
 *                      keys and values into a paged 4-bit cache, and back.
 *   fa_decode_paged_window, fa_decode_paged_q4
 *                      one-token attention over a paged 16-bit or 4-bit cache
 *                      with shared key heads, a sliding window and sinks.
 *   fa_rope            rotary positions of queries and keys, and their gradient.
 *   fa_rope_kv_write   the same on the way into a paged 16-bit cache.
 *   fa_fwd_paged       attention of chunks of new tokens over a paged cache.
 *   fa_kv_weights      the attention weight that each cached key receives.
 *   fa_kv_evict        the keys of least weight leave a paged cache.
 *
 * Common rules
 *   - Every tensor pointer is a DEVICE pointer owned by the caller. The library
 *     allocates no memory and keeps no state between calls, apart from one
 *     device-resident error word per GPU (see fa_check_device_error) and the
 *     test setting of fa_test_withhold_load (off unless a test turns it on).
 *   - Calls are asynchronous: work is enqueued on `stream` (a cudaStream_t
 *     passed as void*, NULL = the legacy default stream) and the call returns
 *     after the launch. Inputs must stay valid until the work completes.
 *   - Arguments are validated on the host before anything is launched; a
 *     failed check returns a negative status and enqueues nothing. Contents of
 *     device arrays (cu_seqlens) are not read on the host.
 *   - 16-bit tensors are contiguous, row-major, 16-byte aligned; fp32 arrays
 *     are contiguous and 4-byte aligned. D is 64 or 128 (the forward also
 *     takes 256, 512 and 1024).
 *   - `scale` multiplies Q K^T before the softmax and must be finite and > 0
 *     (1/sqrt(D) is the usual value).
 *   - LSE outputs are natural-log sums over the scaled, masked scores:
 *     LSE_i = ln sum_j exp(scale * q_i . k_j).
 *   - No C++ exception crosses this boundary.
 *
 * The kernels are compiled for sm_103a only; on another GPU every launch fails
 * with FA_ERR_CUDA.
 */
#ifndef FA_H
#define FA_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FA_API __attribute__((visibility("default")))
#else
#define FA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FA_OK = 0,
    FA_ERR_NULL = -1,           /* a required pointer is NULL */
    FA_ERR_SHAPE = -2,          /* a size is <= 0, or too large for 32-bit indexing, or arrays lie on one another */
    FA_ERR_HEADDIM = -3,        /* D not supported: forward 64/128/256/512/1024, decode and backward 64/128 */
    FA_ERR_DTYPE = -4,          /* dtype is not FA_FP16 or FA_BF16 */
    FA_ERR_ALIGN = -5,          /* a 16-bit tensor is not 16-byte aligned (fp32: 4-byte) */
    FA_ERR_SPLITS = -6,         /* num_splits < 1 or > Sk (or > FA_MAX_SPLITS) */
    FA_ERR_SCALE = -7,          /* scale is not finite and > 0 */
    FA_ERR_CUDA = -8,           /* the CUDA runtime reported an error (launch, tensor map) */
    FA_ERR_DEVICE_TIMEOUT = -9, /* a kernel gave up waiting on an on-chip barrier */
    FA_ERR_SCRATCH = -10,       /* fa_decode_noalloc: problem larger than its built-in scratch */
    FA_ERR_DEVICE_INDEX = -11,  /* a kernel met an out-of-range block-table entry */
    FA_ERR_WORKSPACE = -12,     /* caller workspace smaller than required */
    FA_ERR_DEVICE_SEQLENS = -13 /* fa_fwd_varlen: cu_seqlens inconsistent with the sizes (see there) */
} fa_status_t;

typedef enum { FA_FP16 = 0, FA_BF16 = 1 } fa_dtype_t;

/* Upper bound on the number of KV partitions of the split-KV decode. */
#define FA_MAX_SPLITS 1024

/*
 * fa_fwd - exact attention forward pass, O = softmax(scale * Q K^T [+ mask]) V.
 *
 * Defined by "FlashAttention-2 MMA" (Usage Example: [B,H,S,D] tensors and a
 * causal flag; Technical Details: online softmax with running max and sum,
 * causal rule k_idx <= q_idx) and "Adaptive High-Performance Attention Kernels
 * in CUDA" (Architectural Progression, stages 3-4: outer loop over query
 * tiles, on-chip output accumulator, upper-triangular tiles skipped).
 *
 *   q    [B,H,Sq,D]  fp16/bf16          k, v [B,H,Sk,D]  same dtype
 *   o    [B,H,Sq,D]  output, dtype of q
 *   lse  [B,H,Sq]    fp32 output
 *   causal  0 or 1. When 1, query i sees keys j <= i (top-left alignment,
 *           also when Sq != Sk).
 *   D       64, 128, 256, 512 or 1024. D = 256 covers the pages' large-head
 *           ("GPT-4 style", head_dim 256) configuration and runs a kernel with
 *           one query tile per CTA and 64-key K/V tiles. D = 512 and 1024 (the
 *           pages' "Large Head" and "Massive Head" rows) take the Split-D
 *           strategy ("FlashAttention-2 MMA", Supported Dispatch
 *           Strategies 3: head_dim > 256 partitions the
 *           head dimension across thread blocks): each CTA forms the full
 *           scores and writes one 256-column slice of O. Same results
 *           contract for every D.
 * Errors: FA_ERR_NULL, FA_ERR_SHAPE (B,H,Sq,Sk < 1), FA_ERR_HEADDIM,
 * FA_ERR_DTYPE, FA_ERR_ALIGN, FA_ERR_SCALE, FA_ERR_CUDA.
 */
FA_API fa_status_t fa_fwd(const void *q, const void *k, const void *v, void *o, float *lse,
                   int B, int H, int Sq, int Sk, int D, int causal, float scale,
                   fa_dtype_t dtype, void *stream);

/*
 * fa_fwd_varlen - the forward pass over packed sequences of different lengths.
 *
 * Defined by "Adaptive High-Performance Attention Kernels in CUDA" (Advanced
 * Production Features 3: tokens flattened to [total_tokens, H, d], sequence
 * boundaries from cumulative lengths, no padding computed).
 *
 *   q, o          [total_q,H,D]      k, v [total_k,H,D]
 *   lse           [H,total_q] fp32   (per-head contiguous)
 *   cu_seqlens_q  device int32[num_seqs+1], 0 = cu[0] <= cu[1] <= ... = total_q
 *   cu_seqlens_k  device int32[num_seqs+1], same rules with total_k
 *   max_seqlen_q  >= every query length (sizes the launch)
 * Sequence i attends its own keys only; causal positions are counted from the
 * start of each sequence. Zero-length sequences are allowed. A tile that ends a
 * sequence is multiplied whole, so the up to 127 rows behind it in the tensors
 * must be finite (the window forms below have no such rule).
 * The offsets are checked on the device (the host cannot read them without a
 * synchronisation): if cu_seqlens_q or cu_seqlens_k is negative, decreasing or
 * beyond total_q / total_k, or a query sequence is longer than max_seqlen_q,
 * the launch computes nothing (o and lse are neither read nor written) and
 * the next fa_check_device_error returns FA_ERR_DEVICE_SEQLENS.
 * Errors: as fa_fwd, plus FA_ERR_SHAPE for num_seqs < 1 or total_* < 1.
 */
FA_API fa_status_t fa_fwd_varlen(const void *q, const void *k, const void *v, void *o, float *lse,
                          const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                          int num_seqs, int total_q, int total_k, int max_seqlen_q,
                          int H, int D, int causal, float scale, fa_dtype_t dtype,
                          void *stream);

/*
 * fa_decode_splitkv - split-KV decoding, phase 1 (one query per head).
 *
 * Defined by "Adaptive High-Performance Attention Kernels in CUDA" (Advanced
 * Production Features 1: the KV cache is split into S partitions that run
 * partial attention concurrently) and "FlashAttention-2 MMA" (Split-KV
 * strategy for S_q = 1).
 *
 * Partition s covers keys [s*P, min((s+1)*P, Sk)) with P = ceil(Sk/S); the
 * last partitions may be short or empty. For each (b,h,s):
 *   m_part[b,h,s] = max_j scale * q . k_j                  (-inf if empty)
 *   l_part[b,h,s] = sum_j exp(scale * q . k_j - m)         (0 if empty)
 *   o_part[b,h,s,:] = sum_j exp(scale * q . k_j - m) v_j   (unnormalised)
 *
 *   q [B,H,1,D] (= [B,H,D])   k, v [B,H,Sk,D]   fp16/bf16
 *   o_part [B,H,S,D] fp32, m_part and l_part [B,H,S] fp32: caller workspace.
 * Errors: FA_ERR_NULL, FA_ERR_SHAPE, FA_ERR_HEADDIM, FA_ERR_DTYPE,
 * FA_ERR_ALIGN, FA_ERR_SPLITS, FA_ERR_SCALE, FA_ERR_CUDA.
 */
FA_API fa_status_t fa_decode_splitkv(const void *q, const void *k, const void *v, float *o_part,
                              float *m_part, float *l_part, int B, int H, int Sk, int D,
                              int num_splits, float scale, fa_dtype_t dtype, void *stream);

/*
 * fa_decode_paged_splitkv - split-KV decoding, phase 1, over a paged KV cache.
 *
 * Defined by "Adaptive High-Performance Attention Kernels in CUDA" (Advanced
 * Production Features 4: the KV cache is kept as physical pages
 * [num_blocks, H, block_size, d] and a per-sequence block table translates a
 * logical key position into a page) combined with the split-KV phase 1 above.
 *
 *   q            [B,H,1,D] fp16/bf16
 *   k_cache, v_cache [num_blocks,H,block_size,D], same dtype
 *   block_table  device int32 [B, max_blocks_per_seq]: page of each logical
 *                block; entries past a sequence's length are never read
 *   seq_lens     device int32 [B]: keys of each sequence (clamped to
 *                [0, max_blocks_per_seq * block_size])
 *   o_part [B,H,S,D], m_part and l_part [B,H,S] fp32 outputs, as in
 *                fa_decode_splitkv, with partition size ceil(seq_lens[b]/S)
 *                per sequence (a length-0 sequence has only empty partitions).
 *   block_size   a power of two, 1..1024.
 * Page numbers outside [0, num_blocks) are never dereferenced: their keys are
 * skipped and fa_check_device_error later returns FA_ERR_DEVICE_INDEX.
 * Phase 2 is fa_splitkv_merge, unchanged.
 * Errors: FA_ERR_NULL, FA_ERR_SHAPE, FA_ERR_HEADDIM, FA_ERR_DTYPE,
 * FA_ERR_ALIGN, FA_ERR_SPLITS, FA_ERR_SCALE, FA_ERR_CUDA.
 */
FA_API fa_status_t fa_decode_paged_splitkv(const void *q, const void *k_cache, const void *v_cache,
                                           const int32_t *block_table, const int32_t *seq_lens,
                                           float *o_part, float *m_part, float *l_part, int B, int H,
                                           int D, int num_blocks, int block_size,
                                           int max_blocks_per_seq, int num_splits, float scale,
                                           fa_dtype_t dtype, void *stream);

/*
 * fa_splitkv_merge - split-KV decoding, phase 2 (log-sum-exp reduction).
 *
 * Defined by "Adaptive High-Performance Attention Kernels in CUDA" (Advanced
 * Production Features 1: O = sum_s e^{m_s - m_global} / l_global * O_s), read
 * with m_global = max_s m_s and l_global = sum_s e^{m_s - m_global} l_s.
 *
 *   inputs as written by fa_decode_splitkv with the same B, H, D, num_splits
 *   o   [B,H,1,D] output (dtype)     lse [B,H] fp32 output = m_global + ln l_global
 * Errors: FA_ERR_NULL, FA_ERR_SHAPE, FA_ERR_HEADDIM, FA_ERR_DTYPE,
 * FA_ERR_ALIGN, FA_ERR_SPLITS, FA_ERR_CUDA.
 */
FA_API fa_status_t fa_splitkv_merge(const float *o_part, const float *m_part, const float *l_part,
                             void *o, float *lse, int B, int H, int D, int num_splits,
                             fa_dtype_t dtype, void *stream);

/*
 * fa_decode_splitkv_fused - split-KV decoding, phase 1 and phase 2 in one
 * launch.
 *
 * Computes what fa_decode_splitkv followed by fa_splitkv_merge computes
 * ("Adaptive High-Performance Attention Kernels in CUDA", Advanced Production
 * Features 1: partial attention per partition, then the log-sum-exp merge),
 * without the second launch: each partition's CTA writes its partials to
 * o_part, m_part, l_part (same layout and values as fa_decode_splitkv), then
 * counts itself done on the head's counter; the CTA that finishes last merges
 * the head into o and lse and sets the counter back to zero.
 *
 *   q, k, v, o_part, m_part, l_part, B, H, Sk, D, num_splits, scale, dtype:
 *             as fa_decode_splitkv
 *   o         [B,H,1,D] output (dtype), lse [B,H] fp32: as fa_splitkv_merge
 *   counters  device int32 [B*H], caller-owned. All zero before the first
 *             call; a call that completes leaves it all zero again, so it can
 *             be reused without clearing. If a call fails to launch, clear it.
 * Calls that share counters or partial buffers must not overlap on the GPU.
 * Errors: as fa_decode_splitkv, plus FA_ERR_NULL when o, lse or counters is
 * NULL and FA_ERR_ALIGN when o is not 16-byte or lse/counters not 4-byte
 * aligned.
 */
FA_API fa_status_t fa_decode_splitkv_fused(const void *q, const void *k, const void *v, void *o, float *lse,
                                           float *o_part, float *m_part, float *l_part, int32_t *counters,
                                           int B, int H, int Sk, int D, int num_splits, float scale,
                                           fa_dtype_t dtype, void *stream);

/*
 * fa_decode_paged_splitkv_fused - fa_decode_paged_splitkv and
 * fa_splitkv_merge in one launch, over a paged KV cache ("Adaptive ...",
 * Advanced Production Features 4 and 1).
 *
 *   arguments as fa_decode_paged_splitkv, plus o, lse and counters as
 *   fa_decode_splitkv_fused (same rules for counters).
 * A length-0 sequence gives o = 0 and lse = -inf. Out-of-range page numbers
 * are skipped and reported as by fa_decode_paged_splitkv.
 * Errors: as fa_decode_paged_splitkv, plus those of fa_decode_splitkv_fused
 * for o, lse and counters.
 */
FA_API fa_status_t fa_decode_paged_splitkv_fused(const void *q, const void *k_cache, const void *v_cache,
                                                 const int32_t *block_table, const int32_t *seq_lens, void *o,
                                                 float *lse, float *o_part, float *m_part, float *l_part,
                                                 int32_t *counters, int B, int H, int D, int num_blocks,
                                                 int block_size, int max_blocks_per_seq, int num_splits,
                                                 float scale, fa_dtype_t dtype, void *stream);

/*
 * fa_bwd_workspace_bytes - bytes of workspace fa_bwd needs:
 * 4 * (B*H*Sq*D + 2*B*H*ceil(Sq/128)*128) + 16 (an fp32 dQ accumulator, the
 * per-row statistics and the work counter of the D = 128 kernel); 0 for an
 * invalid shape.
 */
FA_API size_t fa_bwd_workspace_bytes(int B, int H, int Sq, int D);

/*
 * fa_bwd - exact attention backward pass.
 *
 * Defined by "Adaptive High-Performance Attention Kernels in CUDA" (Advanced
 * Production Features 2, Custom CUDA Backward Pass): S = scale Q K^T and
 * P = exp(S - LSE) are recomputed on chip from the forward's LSE (P is never
 * stored), D_i = sum_k dO_ik O_ik, dS = P (dP - D_i) with dP = dO V^T; then
 * dV = P^T dO, dK = scale dS^T Q, dQ = scale dS K (chain rule of the same
 * definition), with the causal rule of fa_fwd.
 *
 *   q, o, dout  [B,H,Sq,D]  fp16/bf16   k, v [B,H,Sk,D]  same dtype
 *   lse         [B,H,Sq] fp32, as written by fa_fwd for these q, k, v
 *   dq [B,H,Sq,D], dk and dv [B,H,Sk,D]: outputs in the input dtype
 *   workspace   caller-owned device memory of at least
 *               fa_bwd_workspace_bytes(B, H, Sq, D) bytes, 16-byte aligned
 *               (fp32 dQ accumulator, per-row statistics, work counter); its
 *               contents on entry do not matter. Calls sharing a workspace
 *               must not overlap on the GPU.
 *   D           64 or 128.
 * Three launches on `stream`. dQ sums contributions of all key tiles with
 * fp32 atomic additions, so its rounding can differ between runs; dK and dV
 * are deterministic.
 * Errors: FA_ERR_NULL, FA_ERR_SHAPE, FA_ERR_HEADDIM, FA_ERR_DTYPE,
 * FA_ERR_ALIGN, FA_ERR_SCALE, FA_ERR_WORKSPACE, FA_ERR_CUDA.
 */
FA_API fa_status_t fa_bwd(const void *q, const void *k, const void *v, const void *o, const void *dout,
                          const float *lse, void *dq, void *dk, void *dv, float *workspace,
                          size_t workspace_bytes, int B, int H, int Sq, int Sk, int D, int causal,
                          float scale, fa_dtype_t dtype, void *stream);

/*
 * fa_bwd_varlen_workspace_bytes - bytes of workspace fa_bwd_varlen needs:
 * 4 * (total_q*H*D + 2*H*total_q) + 16; 0 for an invalid shape.
 */
FA_API size_t fa_bwd_varlen_workspace_bytes(int total_q, int H, int D);

/*
 * fa_bwd_varlen - the backward pass over packed sequences of different lengths.
 *
 * Defined by "Adaptive High-Performance Attention Kernels in CUDA" (Advanced
 * Production Features 2, Custom CUDA Backward Pass, and 3, Ragged / Variable-
 * Length Sequences): the gradients of fa_fwd_varlen. Each sequence is an
 * independent attention over its own keys, so its gradients are those of
 * fa_bwd on that sequence alone; causal positions count from each sequence's
 * start (top-left, as in fa_fwd_varlen). Rows behind a sequence must be finite,
 * as there.
 *
 *   q, o, dout    [total_q,H,D]  fp16/bf16   k, v [total_k,H,D]  same dtype
 *   lse           [H,total_q] fp32, as written by fa_fwd_varlen
 *   dq [total_q,H,D], dk and dv [total_k,H,D]: outputs in the input dtype;
 *                 rows of tokens outside every sequence are left unwritten in
 *                 dk and dv, and dq rows outside every sequence are zero
 *   cu_seqlens_q, cu_seqlens_k   device int32[num_seqs+1], as in fa_fwd_varlen
 *   max_seqlen_q, max_seqlen_k   >= every query / key length (size the launch)
 *   workspace     caller-owned device memory of at least
 *                 fa_bwd_varlen_workspace_bytes(total_q, H, D) bytes, 16-byte
 *                 aligned; its contents on entry do not matter. Calls sharing
 *                 a workspace must not overlap on the GPU.
 *   D             64 or 128.
 * Keys of a sequence without queries get dK = dV = 0. Three launches on
 * `stream`; dQ's fp32 additions make its rounding run-dependent, dK and dV are
 * deterministic. The offsets are checked on the device: a sequence whose
 * offsets lie outside the tensors, or that is longer than max_seqlen_q /
 * max_seqlen_k, is skipped (its gradients are not written) and the next
 * fa_check_device_error returns FA_ERR_DEVICE_SEQLENS.
 * Errors: FA_ERR_NULL, FA_ERR_SHAPE, FA_ERR_HEADDIM, FA_ERR_DTYPE,
 * FA_ERR_ALIGN, FA_ERR_SCALE, FA_ERR_WORKSPACE, FA_ERR_CUDA.
 */
FA_API fa_status_t fa_bwd_varlen(const void *q, const void *k, const void *v, const void *o, const void *dout,
                                 const float *lse, void *dq, void *dk, void *dv, float *workspace,
                                 size_t workspace_bytes, const int32_t *cu_seqlens_q,
                                 const int32_t *cu_seqlens_k, int num_seqs, int total_q, int total_k,
                                 int max_seqlen_q, int max_seqlen_k, int H, int D, int causal, float scale,
                                 fa_dtype_t dtype, void *stream);

/*
 * fa_fwd_window - fa_fwd with a sliding window, sinks and shared key heads.
 *
 * Query i sees key j if j <= i (top-left, as fa_fwd's causal rule) and either
 * i - j < window or j < sinks: its own key and the window - 1 before it, and
 * the first `sinks` keys. window >= 1, sinks >= 0; a window of Sq or more is
 * plain causal attention. Key tiles that no query of a tile sees are not read,
 * so the work grows with Sq * (window + sinks). Query 0 is at position 0: there
 * is no offset for queries that come behind a cached prefix (their prefix's
 * queries are passed too, or the new tokens decoded one by one).
 *
 *   q, o [B,H,Sq,D], lse [B,H,Sq], k, v [B,Hkv,Sk,D] as in fa_fwd; query head
 *   h reads key head h / (H / Hkv); Hkv divides H; D is 64 or 128.
 * A query that sees no key (Sq > Sk, beyond the window) gets o = 0 and
 * lse = -inf. Hidden keys and values must be finite: a tile that a query sees
 * in part is multiplied whole, with zero weights.
 * Errors: as fa_fwd; FA_ERR_SHAPE also when Hkv does not divide H, window < 1,
 * sinks < 0, or a length is above 2^29.
 */
FA_API fa_status_t fa_fwd_window(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H,
                                 int Hkv, int Sq, int Sk, int D, int window, int sinks, float scale,
                                 fa_dtype_t dtype, void *stream);

/*
 * fa_fwd_window_varlen - fa_fwd_window over packed sequences: arguments and
 * device-side checks as fa_fwd_varlen (positions, the window and the sinks
 * count from each sequence's start), k and v [total_k,Hkv,D]. Hidden keys and
 * values of a sequence itself must be finite, as there; rows that are not its
 * own may hold anything, NaNs included.
 * Errors: as fa_fwd_varlen and fa_fwd_window.
 */
FA_API fa_status_t fa_fwd_window_varlen(const void *q, const void *k, const void *v, void *o, float *lse,
                                        const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int num_seqs,
                                        int total_q, int total_k, int max_seqlen_q, int H, int Hkv, int D,
                                        int window, int sinks, float scale, fa_dtype_t dtype, void *stream);

/*
 * fa_bwd_window_workspace_bytes, fa_bwd_window_varlen_workspace_bytes - bytes
 * of workspace that fa_bwd_window and fa_bwd_window_varlen need: those of
 * fa_bwd (fa_bwd_varlen), and 1024 D bytes (fp32 dV and dK of 128 keys) for
 * each segment into which the work of a key tile is cut where shared heads or
 * sinks make it long. 0 for an invalid shape.
 */
FA_API size_t fa_bwd_window_workspace_bytes(int B, int H, int Hkv, int Sq, int Sk, int D, int window, int sinks);
FA_API size_t fa_bwd_window_varlen_workspace_bytes(int num_seqs, int total_q, int max_seqlen_q, int max_seqlen_k,
                                                   int H, int Hkv, int D, int window, int sinks);

/*
 * fa_bwd_window - the gradients of fa_fwd_window, as fa_bwd computes those of
 * fa_fwd: dq [B,H,Sq,D], and dk, dv [B,Hkv,Sk,D] summed over the query heads
 * that share a key head. workspace: at least fa_bwd_window_workspace_bytes
 * bytes, otherwise as for fa_bwd. Queries that see no key get dq = 0, keys that
 * no query sees dk = dv = 0. dk and dv are deterministic, dq rounds as in
 * fa_bwd. Three launches.
 * Errors: as fa_bwd and fa_fwd_window.
 */
FA_API fa_status_t fa_bwd_window(const void *q, const void *k, const void *v, const void *o, const void *dout,
                                 const float *lse, void *dq, void *dk, void *dv, float *workspace,
                                 size_t workspace_bytes, int B, int H, int Hkv, int Sq, int Sk, int D, int window,
                                 int sinks, float scale, fa_dtype_t dtype, void *stream);

/*
 * fa_bwd_window_varlen - the gradients of fa_fwd_window_varlen: arguments,
 * device-side checks and rows outside the sequences as fa_bwd_varlen, the
 * workspace of fa_bwd_window_varlen_workspace_bytes, dk and dv [total_k,Hkv,D].
 * As in the forward, rows that are not a sequence's own (of q, k, v, o, dout and
 * lse) may hold anything.
 * Errors: as fa_bwd_varlen and fa_fwd_window.
 */
FA_API fa_status_t fa_bwd_window_varlen(const void *q, const void *k, const void *v, const void *o, const void *dout,
                                        const float *lse, void *dq, void *dk, void *dv, float *workspace,
                                        size_t workspace_bytes, const int32_t *cu_seqlens_q,
                                        const int32_t *cu_seqlens_k, int num_seqs, int total_q, int total_k,
                                        int max_seqlen_q, int max_seqlen_k, int H, int Hkv, int D, int window,
                                        int sinks, float scale, fa_dtype_t dtype, void *stream);

/*
 * The paged 4-bit cache of keys and values (fa_kv_write_q4, fa_kv_read_q4,
 * fa_decode_paged_q4). Keys and values are held alike, each as two arrays:
 *
 *   codes   uint8   [num_blocks, Hkv, block_size, D / 2]
 *   scales  fp16/bf16 [num_blocks, Hkv, block_size, D / FA_Q4_GROUP]
 *
 * FA_Q4_GROUP = 32 consecutive columns of a row share a scale
 *   s = max|x| / 7, rounded to the 16-bit type (nearest, ties to even), and
 *   n = x / s rounded to the nearest integer (ties to even), within [-7, 7];
 * a group whose s rounds to zero has n = 0. The cache stands for s * n. A
 * group that holds an infinity or a NaN gets s = NaN and stands for NaNs.
 * Column d = 32 w + 4 g + i (g < 8, i < 4) of a row is held as n + 8 in nibble
 * i % 2 (0: bits 0-3) of byte g * (D / 16) + 2 w + i / 2 of the row.
 */
#define FA_Q4_GROUP 32

/*
 * fa_kv_write_q4 - quantise new keys and values and store them in the cache.
 *
 *   k, v         [total,Hkv,D] fp16/bf16, the new tokens of all sequences,
 *                packed; D is 64 or 128
 *   k_codes, k_scales, v_codes, v_scales   the cache (see above), scales in
 *                the dtype of k and v; only the rows of the new tokens change
 *   block_table  device int32 [num_seqs, max_blocks_per_seq]: page of each
 *                logical block of a sequence
 *   cu_seqlens   device int32 [num_seqs + 1], 0 <= cu[0] <= cu[1] <= ... <=
 *                total: sequence b's new tokens are rows [cu[b], cu[b+1])
 *   starts       device int32 [num_seqs]: position in its sequence of the
 *                first new token of each sequence (>= 0), or NULL: all zero
 *   max_seqlen   >= every number of new tokens (sizes the launch)
 *   block_size   a power of two, 1..1024
 * Position p of sequence b is row p % block_size of page
 * block_table[b][p / block_size]. Two tokens of one call must not fall on the
 * same row of the same page (each group of such a row ends up as either's).
 * A sequence whose offsets do not fit [0, total] and max_seqlen, or whose
 * start is negative, is skipped and the next fa_check_device_error returns
 * FA_ERR_DEVICE_SEQLENS; a position past max_blocks_per_seq * block_size or a
 * page number outside [0, num_blocks) is skipped and reported as
 * FA_ERR_DEVICE_INDEX. total = 0 is allowed (max_seqlen may then be 0) and
 * does nothing.
 * Errors: FA_ERR_NULL, FA_ERR_SHAPE, FA_ERR_HEADDIM, FA_ERR_DTYPE,
 * FA_ERR_ALIGN, FA_ERR_CUDA.
 */
FA_API fa_status_t fa_kv_write_q4(const void *k, const void *v, void *k_codes, void *k_scales, void *v_codes,
                                  void *v_scales, const int32_t *block_table, const int32_t *cu_seqlens,
                                  const int32_t *starts, int num_seqs, int total, int max_seqlen, int Hkv, int D,
                                  int num_blocks, int block_size, int max_blocks_per_seq, fa_dtype_t dtype,
                                  void *stream);

/*
 * fa_kv_read_q4 - read stretches of the cache back as 16-bit keys and values
 * (s * n rounded to the 16-bit type), packed as fa_fwd_varlen and
 * fa_fwd_window_varlen take them.
 *
 *   k, v         [total,Hkv,D] outputs, dtype of the scales; rows outside
 *                every sequence, and rows that are skipped, are left as they
 *                were (fa_fwd_varlen wants finite values there)
 *   all other arguments as fa_kv_write_q4: row cu[b] + i receives position
 *   starts[b] + i of sequence b.
 * Offsets, positions and page numbers are checked on the device as by
 * fa_kv_write_q4.
 * Errors: as fa_kv_write_q4.
 */
FA_API fa_status_t fa_kv_read_q4(void *k, void *v, const void *k_codes, const void *k_scales, const void *v_codes,
                                 const void *v_scales, const int32_t *block_table, const int32_t *cu_seqlens,
                                 const int32_t *starts, int num_seqs, int total, int max_seqlen, int Hkv, int D,
                                 int num_blocks, int block_size, int max_blocks_per_seq, fa_dtype_t dtype,
                                 void *stream);

/*
 * fa_decode_splits - a number of partitions for fa_decode_paged_window and
 * fa_decode_paged_q4 that is fast on the current GPU: it fills the GPU, but for
 * few heads of sequences too short to repay the joining of so many parts. For a
 * batch of B sequences, Hkv key heads and at most max_keys visible keys a
 * sequence (window + sinks, or the longest sequence). At least 1, at most
 * FA_MAX_SPLITS; 1 where the arguments are not positive.
 */
FA_API int fa_decode_splits(int B, int H, int Hkv, int max_keys);

/*
 * fa_decode_paged_window - attention of one new token per sequence over a
 * paged cache, with shared key heads, a sliding window and sinks, in one
 * launch: split-KV decoding as fa_decode_paged_splitkv_fused does it, over the
 * keys that the token sees.
 *
 * The query is at position L - 1 of a sequence of L = seq_lens[b] keys (its
 * own key is in the cache) and sees key j if L - 1 - j < window, or window is
 * 0 (all keys), or j < sinks.
 *
 *   q            [B,H,1,D] fp16/bf16; query head h reads key head
 *                h / (H / Hkv); Hkv divides H; D is 64 or 128
 *   k_cache, v_cache [num_blocks,Hkv,block_size,D], same dtype
 *   block_table  device int32 [B, max_blocks_per_seq]; entries whose keys are
 *                not visible are never read
 *   seq_lens     device int32 [B] (clamped to [0, max_blocks_per_seq *
 *                block_size]); a length of 0 gives o = 0 and lse = -inf
 *   o [B,H,1,D] (dtype), lse [B,H] fp32: outputs
 *   o_part       [B,H,num_splits,D], m_part and l_part [B,H,num_splits] fp32:
 *                workspace (the visible keys of a sequence are cut into up to
 *                num_splits partitions); contents on entry and exit mean
 *                nothing
 *   counters     device int32 [B*H]: all zero before the first call, left all
 *                zero by every completed call
 *   window >= 0, sinks >= 0; block_size a power of two, 1..1024
 * Rows of a page that the token does not see may hold anything, NaNs
 * included. Page numbers outside [0, num_blocks) are not dereferenced: their
 * keys are skipped and fa_check_device_error returns FA_ERR_DEVICE_INDEX.
 * Calls that share counters or partial buffers must not overlap on the GPU.
 * Errors: FA_ERR_NULL, FA_ERR_SHAPE (Hkv does not divide H; window or sinks
 * negative; sizes), FA_ERR_HEADDIM, FA_ERR_DTYPE, FA_ERR_ALIGN (o_part too is
 * 16-byte aligned), FA_ERR_SPLITS, FA_ERR_SCALE, FA_ERR_CUDA.
 */
FA_API fa_status_t fa_decode_paged_window(const void *q, const void *k_cache, const void *v_cache,
                                          const int32_t *block_table, const int32_t *seq_lens, void *o, float *lse,
                                          float *o_part, float *m_part, float *l_part, int32_t *counters, int B,
                                          int H, int Hkv, int D, int num_blocks, int block_size,
                                          int max_blocks_per_seq, int num_splits, int window, int sinks,
                                          float scale, fa_dtype_t dtype, void *stream);

/*
 * fa_decode_paged_q4 - fa_decode_paged_window over the 4-bit cache: the keys
 * and values are s * n, not rounded to 16 bits. Scales have the dtype of q.
 * Arguments, rules and errors as fa_decode_paged_window, with the cache of
 * fa_kv_write_q4 in place of k_cache and v_cache.
 */
FA_API fa_status_t fa_decode_paged_q4(const void *q, const void *k_codes, const void *k_scales, const void *v_codes,
                                      const void *v_scales, const int32_t *block_table, const int32_t *seq_lens,
                                      void *o, float *lse, float *o_part, float *m_part, float *l_part,
                                      int32_t *counters, int B, int H, int Hkv, int D, int num_blocks,
                                      int block_size, int max_blocks_per_seq, int num_splits, int window, int sinks,
                                      float scale, fa_dtype_t dtype, void *stream);

/*
 * fa_rope - rotary positions, or (inverse) their gradient.
 *
 * Of each row of D columns the first rot_dim are rot_dim / 2 pairs: columns i
 * and i + rot_dim / 2 (interleaved = 0) or 2 i and 2 i + 1 (interleaved = 1).
 * Pair i, (a, b), of a token at position p becomes
 *   mscale * (a cos t - b sin t, b cos t + a sin t),   t = p * inv_freq[i],
 * rounded once; columns from rot_dim on are copied. inverse = 1 takes -t: the
 * gradient with respect to x, given that of y. Frequencies scaled for long
 * contexts are other values of inv_freq and mscale.
 *
 *   x, y       rows of D fp16/bf16 columns, row (b, s, h) at element
 *              b * x_batch + s * x_token + h * x_head of x, and alike of y:
 *              [B,S,H,D], [B,H,S,D], packed tokens (B = 1, S = total) or a part
 *              of a wider tensor. Strides are >= 0 and multiples of 8. y may be
 *              x itself with the same strides (with others the call is refused);
 *              otherwise they must not overlap, nor may y's rows each other.
 *   inv_freq   device fp32 [rot_dim / 2]; an infinite or NaN one makes its pair
 *              of columns NaN, at position 0 too
 *   positions  device int32 [B,S], or NULL: 0 .. S - 1. Any values: an angle is
 *              formed as a 64-bit fraction of a turn, so far positions keep
 *              theirs (off by 2^-63 |p| max(1, inv_freq / 4) turns at most,
 *              besides 2^-24 of it).
 *   D          64, 128, 256, 512 or 1024; rot_dim a multiple of 16, 16 .. D
 * S = 0 is allowed and does nothing. One launch.
 * Errors: FA_ERR_NULL, FA_ERR_SHAPE (rot_dim and strides too), FA_ERR_HEADDIM,
 * FA_ERR_DTYPE, FA_ERR_ALIGN, FA_ERR_SCALE (mscale is not finite), FA_ERR_CUDA.
 */
FA_API fa_status_t fa_rope(const void *x, void *y, const float *inv_freq, const int32_t *positions, int B, int S,
                           int H, int D, int rot_dim, int64_t x_batch, int64_t x_token, int64_t x_head,
                           int64_t y_batch, int64_t y_token, int64_t y_head, int interleaved, int inverse,
                           float mscale, fa_dtype_t dtype, void *stream);

/*
 * fa_rope_kv_write - new tokens into a paged 16-bit cache, queries and keys
 * rotated on the way (as fa_rope does it), in one launch.
 *
 *   q, q_out     [total,H,D] queries and where they go, rotated; q_out is
 *                contiguous and may be q where that is too (refused where it is
 *                not). H = 0: no queries (both may be NULL).
 *   k, v         [total,Hkv,D]: the new tokens' keys (stored rotated) and
 *                values (stored as they are); D is 64 or 128
 *   q_token, k_token, v_token   elements between tokens of q, k and v (H * D,
 *                Hkv * D for contiguous ones; parts of a joint projection are
 *                wider); multiples of 8
 *   k_cache, v_cache [num_blocks,Hkv,block_size,D], as fa_decode_paged_window
 *                and fa_fwd_paged read them; only the new tokens' rows change
 *   inv_freq     device fp32 [rot_dim / 2]; rot_dim = 0 rotates nothing
 *                (inv_freq may be NULL)
 *   positions    device int32 [total]: rotary position of each packed token, or
 *                NULL: its position in its sequence's cache, starts[b] + i. They
 *                differ once keys have been evicted.
 *   block_table, cu_seqlens, starts, max_seqlen, block_size: as fa_kv_write_q4
 * Offsets, positions in the cache and page numbers are checked on the device as
 * by fa_kv_write_q4 (queries of a token without a page are still rotated).
 * total = 0 is allowed (max_seqlen may then be 0) and does nothing.
 * Errors: FA_ERR_NULL, FA_ERR_SHAPE, FA_ERR_HEADDIM, FA_ERR_DTYPE,
 * FA_ERR_ALIGN, FA_ERR_SCALE (mscale is not finite), FA_ERR_CUDA.
 */
FA_API fa_status_t fa_rope_kv_write(const void *q, const void *k, const void *v, void *q_out, void *k_cache,
                                    void *v_cache, const float *inv_freq, const int32_t *positions,
                                    const int32_t *block_table, const int32_t *cu_seqlens, const int32_t *starts,
                                    int num_seqs, int total, int max_seqlen, int H, int Hkv, int D, int rot_dim,
                                    int64_t q_token, int64_t k_token, int64_t v_token, int num_blocks,
                                    int block_size, int max_blocks_per_seq, int interleaved, float mscale,
                                    fa_dtype_t dtype, void *stream);

/*
 * fa_fwd_paged_workspace_bytes - bytes of workspace fa_fwd_paged needs on the
 * current GPU (two fp32 parts of up to 256 rows of queries for each SM: 40 MB
 * at D = 128, 2.5 MB where a chunk is 16 rows); 0 for an invalid shape.
 */
FA_API size_t fa_fwd_paged_workspace_bytes(int max_seqlen_q, int H, int Hkv, int D);

/*
 * fa_fwd_paged - attention of a chunk of new tokens of each sequence over a
 * paged cache that holds their keys already: a prompt's next piece, drafted
 * tokens, or a serving batch of both and single tokens.
 *
 * The last query of a sequence is at its last key: query t of Lq is at position
 * p = L - Lq + t of L = seq_lens[b] keys, and sees key j if j <= p and
 * (p - j < window, or window is 0, or j < sinks).
 *
 *   q, o         [total_q,H,D] fp16/bf16, the chunks packed; query head h reads
 *                key head h / (H / Hkv); Hkv divides H, into groups of at most
 *                128; D is 64 or 128
 *   k_cache, v_cache [num_blocks,Hkv,block_size,D], same dtype, as
 *                fa_rope_kv_write fills them
 *   block_table  device int32 [num_seqs, max_blocks_per_seq]; entries whose
 *                keys no query sees are never read
 *   cu_seqlens_q device int32 [num_seqs + 1], 0 <= cu[0] <= cu[1] <= ... <=
 *                total_q: sequence b's chunk is rows [cu[b], cu[b+1])
 *   seq_lens     device int32 [num_seqs]: keys of each sequence, its chunk's
 *                among them (clamped to [0, max_blocks_per_seq * block_size])
 *   lse          [H,total_q] fp32 output
 *   workspace    caller-owned, at least fa_fwd_paged_workspace_bytes bytes,
 *                16-byte aligned; contents on entry and exit mean nothing. Calls
 *                that share one must not overlap on the GPU.
 *   max_seqlen_q >= every chunk's length; window, sinks >= 0
 *   block_size   a power of two, 1..1024. Pages of 8 rows and more are loaded
 *                as tiles; smaller ones are slower.
 * A query that sees no key (more queries than keys) gets o = 0 and lse = -inf.
 * Rows of o and lse that belong to no chunk are left as they were. Rows of a page
 * that no query sees may hold anything, NaNs included; the others must be finite
 * (a key tile is multiplied whole, hidden keys with zero weights).
 * The softmax weights are rounded to the 16-bit type before they meet V, as in
 * fa_fwd: o is off by 2.3e-3 of itself in bf16 (2.7e-4 in fp16), root mean square,
 * where its own rounding alone is 1.7e-3 (2.1e-4). fa_decode_paged_window does not
 * round them so and is nearer to that.
 * `window` counts places in the cache. Behind fa_kv_evict, whose key heads each
 * keep keys of their own, that is no longer a distance in tokens.
 * Offsets outside [0, total_q], decreasing ones, or a chunk longer than
 * max_seqlen_q: nothing is computed and the next fa_check_device_error returns
 * FA_ERR_DEVICE_SEQLENS. Page numbers outside [0, num_blocks) are not
 * dereferenced: their rows count as zeros, and it returns FA_ERR_DEVICE_INDEX.
 * The result is deterministic. Two launches.
 * Errors: FA_ERR_NULL, FA_ERR_SHAPE, FA_ERR_HEADDIM, FA_ERR_DTYPE,
 * FA_ERR_ALIGN, FA_ERR_SCALE, FA_ERR_WORKSPACE, FA_ERR_CUDA.
 */
FA_API fa_status_t fa_fwd_paged(const void *q, const void *k_cache, const void *v_cache, const int32_t *block_table,
                                const int32_t *cu_seqlens_q, const int32_t *seq_lens, void *o, float *lse,
                                float *workspace, size_t workspace_bytes, int num_seqs, int total_q,
                                int max_seqlen_q, int H, int Hkv, int D, int num_blocks, int block_size,
                                int max_blocks_per_seq, int window, int sinks, float scale, fa_dtype_t dtype,
                                void *stream);

/*
 * fa_kv_weights - what a chunk of queries gave to each key of a paged cache: the
 * softmax weights of the attention that has run, summed over the chunk's
 * queries and the query heads of a key head, and (add = 1) added to what is there
 * or (add = 0) put there:
 *
 *   weights[b, hk, j] (+)= sum over queries t that see key j, and heads h of key
 *                          head hk, of exp(scale * q_th . k_j - lse_th)
 *
 * fa_kv_evict takes them. What a query sees is as in fa_fwd_paged, whose
 * arguments these are, but for
 *
 *   lse        fp32, of the attention over the same keys: (head h, packed token
 *              t) at element h * lse_head + t * lse_token: (total_q, 1) for the
 *              [H,total_q] of fa_fwd_paged, (1, H) for the [B,H] of a decode
 *              (total_q = B queries, one each)
 *   weights    [num_seqs,Hkv,max_blocks_per_seq * block_size] fp32, in and out:
 *              keys that no query sees keep theirs (add = 1) or get zeros, those
 *              behind a sequence too (add = 0)
 * Queries with lse = -inf give nothing. Rows of the cache that no query sees, and
 * rows of q and lse that belong to no chunk, may hold anything. Offsets and page
 * numbers are checked as by fa_fwd_paged (a page that does not exist counts as
 * zeros). The result is deterministic. One launch, no workspace.
 * Sums are fp32: of n terms (queries times heads of a group) a key has eight
 * running ones, so a weight is off by about 2^-27 n of itself at most (1e-7 to
 * 2.5e-7, root mean square, in practice) besides what a term is off by (some
 * 2^-22 (1 + |scale q.k| + |lse|)). With add = 1 a call's sum is rounded to the
 * steps of what is there: below 2^-25 of it, it vanishes.
 * Errors: FA_ERR_NULL, FA_ERR_SHAPE (negative strides too), FA_ERR_HEADDIM,
 * FA_ERR_DTYPE, FA_ERR_ALIGN, FA_ERR_SCALE, FA_ERR_CUDA.
 */
FA_API fa_status_t fa_kv_weights(const void *q, const float *lse, const void *k_cache, const int32_t *block_table,
                                 const int32_t *cu_seqlens_q, const int32_t *seq_lens, float *weights,
                                 int64_t lse_head, int64_t lse_token, int num_seqs, int total_q, int max_seqlen_q,
                                 int H, int Hkv, int D, int num_blocks, int block_size, int max_blocks_per_seq,
                                 int window, int sinks, int add, float scale, fa_dtype_t dtype, void *stream);

/*
 * fa_kv_evict - the keys of least weight leave a paged 16-bit cache.
 *
 * Of a sequence of L = seq_lens[b] keys with L > keep, each key head keeps
 * `keep`: the first `sinks`, the last `recent`, and of those between them the
 * ones of greatest weight (ties to the earlier key; a NaN is less than any
 * number). They keep their order and become keys 0 .. keep - 1 of the new
 * pages, each head its own. With L <= keep all stay, as keys 0 .. L - 1. (A
 * window of a later call counts these places, not tokens.)
 *
 *   k_cache, v_cache [num_blocks,Hkv,block_size,D] fp16/bf16, D 64 or 128
 *   weights      [B,Hkv,max_blocks_per_seq * block_size] fp32, as fa_kv_weights
 *                fills it; not changed
 *   block_table  device int32 [B, max_blocks_per_seq]: the sequences' pages,
 *                which are only read (they may be shared with other sequences)
 *   seq_lens     device int32 [B], clamped as by fa_decode_paged_window
 *   new_table    device int32 [B, new_max_blocks_per_seq]: the pages that the
 *                kept keys go to, none of them a page that the call reads or
 *                names twice. Their rows behind the kept keys are not written.
 *   kept         int32 [B,Hkv,keep] output: what each new key was before
 *                (-1 behind the last one)
 *   new_lens     int32 [B] output: min(L, keep)
 *   new_weights  [B,Hkv,new_max_blocks_per_seq * block_size] fp32 output: the
 *                kept keys' weights, then zeros
 *   Outputs must not overlap the inputs (new_lens is not seq_lens itself,
 *   new_weights not weights) or one another, and new_table is not block_table:
 *   such calls are refused with FA_ERR_SHAPE.
 *   block_size a power of two, 1..1024; keep >= 1, sinks, recent >= 0,
 *   sinks + recent <= keep
 * A key whose old or new page is outside [0, num_blocks), or that has no place
 * in new_table, is not copied and the next fa_check_device_error returns
 * FA_ERR_DEVICE_INDEX. Two launches.
 * Errors: FA_ERR_NULL, FA_ERR_SHAPE, FA_ERR_HEADDIM, FA_ERR_DTYPE,
 * FA_ERR_ALIGN, FA_ERR_CUDA.
 */
FA_API fa_status_t fa_kv_evict(void *k_cache, void *v_cache, const float *weights, const int32_t *block_table,
                               const int32_t *seq_lens, const int32_t *new_table, int32_t *kept, int32_t *new_lens,
                               float *new_weights, int B, int Hkv, int D, int num_blocks, int block_size,
                               int max_blocks_per_seq, int new_max_blocks_per_seq, int keep, int sinks, int recent,
                               fa_dtype_t dtype, void *stream);

/*
 * fa_check_device_error - synchronise `stream`, then read and clear the
 * current device's error word. Kernels bound every wait on an on-chip barrier;
 * a wait that runs out sets the word, releases what the CTA holds and returns.
 * Returns FA_OK, FA_ERR_DEVICE_TIMEOUT, FA_ERR_DEVICE_INDEX (an out-of-range
 * block-table entry was skipped), FA_ERR_DEVICE_SEQLENS (a packed-sequence
 * launch found inconsistent cu_seqlens: see fa_fwd_varlen, fa_bwd_varlen), or FA_ERR_CUDA
 * when the runtime itself reports an error, or a kernel was not given the
 * shared memory that it declares (a base of 1024 bytes' alignment: fa_kv_weights
 * then computes nothing).
 */
FA_API fa_status_t fa_check_device_error(void *stream);

/*
 * fa_test_withhold_load - test support for the failure path of the prefill
 * kernels (fa_fwd, fa_fwd_varlen, fa_bwd, fa_bwd_varlen, the window forms,
 * fa_fwd_paged and fa_kv_weights).
 * With load = n > 0, the CTA with the first work item of every later launch of
 * those kernels never issues one of its tile loads (the forward's V tile
 * n - 1, the backward's Q/dO step n - 1, the query tile n - 1 of fa_kv_weights;
 * an item with n of them), so the
 * wait for it cannot complete: the kernel's bounded wait runs out after
 * `wait_limit_ns`, its CTAs drain the copies they issued, release tensor
 * memory and stop, and fa_check_device_error returns FA_ERR_DEVICE_TIMEOUT.
 * Outputs of such a launch are undefined. `wait_limit_ns` (0 = the default,
 * one second) bounds every on-chip wait of every launch of those kernels.
 * load = 0 and wait_limit_ns = 0 restore normal operation. The setting is
 * process-wide; it is not meant to be changed while other threads launch.
 * Returns FA_OK, or FA_ERR_SHAPE for a negative load.
 */
FA_API fa_status_t fa_test_withhold_load(int load, unsigned long long wait_limit_ns);

/*
 * fa_decode_noalloc - split-KV decoding (phase 1 and phase 2 in one call) that
 * allocates nothing and needs no caller workspace. The pages have no
 * counterpart: this entry point exists for callers that cannot allocate
 * device memory when they call in (an engine hook that must not allocate, a
 * latency-critical loop that cannot take the device-wide synchronisation an
 * allocation may bring, a process whose memory a pool has fully reserved).
 *
 * The partials live in a fixed device array built into the library, of
 * FA_NOALLOC_SCRATCH_FLOATS floats (8 MiB), which every GPU that loads the
 * library holds until the process exits. A call needs
 * B*H*num_splits*D + 2*B*H*num_splits floats (each part rounded up to 4);
 * larger problems return FA_ERR_SCRATCH before anything is enqueued. The
 * first call on a device looks up the array's device address (with that
 * device current); make it before any stream capture. All calls share the
 * array: calls whose work overlaps on the GPU race and must be serialised by
 * the caller. Nothing needs clearing between calls.
 *
 *   q [B,H,1,D], k and v [B,H,Sk,D], o [B,H,1,D] (dtype), lse [B,H] fp32.
 *   Results equal fa_decode_splitkv followed by fa_splitkv_merge.
 * Errors: as fa_decode_splitkv, plus FA_ERR_SCRATCH.
 */
#define FA_NOALLOC_SCRATCH_FLOATS (2 * 1024 * 1024)
FA_API fa_status_t fa_decode_noalloc(const void *q, const void *k, const void *v, void *o, float *lse,
                                     int B, int H, int Sk, int D, int num_splits, float scale,
                                     fa_dtype_t dtype, void *stream);

/* Static, NUL-terminated description of a status code (never NULL). */
FA_API const char *fa_status_string(fa_status_t status);

/* Library version as major*10000 + minor*100 + patch. */
FA_API int fa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_H */
