// C ABI of libfa.so (declared in include/fa.h): argument validation, TMA tensor
// map encoding and kernel launches. Allocates no memory; the only state is one
// device-resident error word per GPU.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <atomic>
#include <mutex>

#include "fa.h"
#include "fa_launch.h"

namespace {

__device__ int g_device_error_word = 0;

constexpr int kMaxDevices = 64;

// Address of the error word on the current device (looked up once per device).
// Test support (fa_test_withhold_load): the load to withhold and the wait
// limit every launch uses.
std::atomic<int> g_withhold{0};
std::atomic<unsigned long long> g_wait_limit_ns{fa::kWaitTimeoutNs};

int *device_error_word() {
    static std::mutex mu;
    static int *cache[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev] == nullptr) {
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_device_error_word) != cudaSuccess) return nullptr;
        cache[dev] = static_cast<int *>(p);
    }
    return cache[dev];
}

int num_sms() {
    static std::mutex mu;
    static int cache[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        cache[dev] = n;
    }
    return cache[dev];
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// 3-D map over a 16-bit tensor whose innermost dimension is D, with 64 x 1 x
// 128 or 64 x 128 x 1 boxes and 128-byte swizzle (rows of 128 bytes land in
// shared memory in the layout the MMA descriptors describe). Out-of-range
// rows read as zero.
bool encode_map(CUtensorMap *m, bool bf16, const void *base, uint64_t d0, uint64_t d1, uint64_t d2,
                uint64_t stride1_bytes, uint64_t stride2_bytes, uint32_t box1, uint32_t box2) {
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {d0, d1, d2};
    const cuuint64_t strides[2] = {stride1_bytes, stride2_bytes};
    const cuuint32_t box[3] = {64, box1, box2};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                          const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// 3-D map over an fp32 dQ accumulator with 32-column boxes and 128-byte
// swizzle: the target of the backward pass's bulk reductions. Dense
// [B*H][Sq][D]: dims {D, Sq, B*H}, boxes 32 x rows x 1; packed [T][H][D]:
// dims {D, H, T}, boxes 32 x 1 x rows.
bool encode_map_f32(CUtensorMap *m, void *base, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t stride1_bytes,
                    uint64_t stride2_bytes, uint32_t box1, uint32_t box2) {
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {d0, d1, d2};
    const cuuint64_t strides[2] = {stride1_bytes, stride2_bytes};
    const cuuint32_t box[3] = {32, box1, box2};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Work units per group of the backward's CTA order: the group's Q, dO and fp32
// dQ accumulator rows (8 L D bytes per unit of L query rows) within 32 MB, a
// quarter of L2.
int bwd_units_per_group(long long units, long long rows, int D) {
    const long long per_unit = 8LL * (rows > 0 ? rows : 1) * D;
    const long long g = (32LL << 20) / per_unit;
    return static_cast<int>(g < 1 ? 1 : (g > units ? units : g));
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool scale_ok(float s) { return std::isfinite(s) && s > 0.f; }

constexpr float kLog2e = 1.4426950408889634f;

// Forward head dimensions: 64 and 128 (two query tiles per work item), 256
// (one), 512 and 1024 (Split-D: one query tile and 256 output columns).
bool fwd_head_dim_ok(int D) { return D == 64 || D == 128 || D == 256 || D == 512 || D == 1024; }

long long fwd_work_items(int D, long long heads, int Sq) {
    const long long n_qtiles = (Sq + 127) / 128;
    if (D >= 256) return heads * n_qtiles * (D / 256);
    return heads * ((n_qtiles + 1) / 2);
}
constexpr int kMaxLen = 1 << 30;
constexpr int kMaxWindowLen = 1 << 29;  // window functions: key + window stays within 32 bits

// Page geometry of a paged cache: block_size a power of two up to 1024, and
// positions and (page, head) indices within 32 bits.
bool pages_ok(int Hkv, int num_blocks, int block_size, int max_blocks, int &log2_bs) {
    if (num_blocks < 1 || max_blocks < 1) return false;
    if (block_size < 1 || block_size > 1024 || (block_size & (block_size - 1)) != 0) return false;
    if (static_cast<long long>(max_blocks) * block_size > kMaxLen) return false;
    if (static_cast<long long>(num_blocks) * Hkv > INT_MAX) return false;
    log2_bs = 0;
    while ((1 << log2_bs) < block_size) ++log2_bs;
    return true;
}

}  // namespace

extern "C" {

int fa_version(void) { return 200; }

const char *fa_status_string(fa_status_t s) {
    switch (s) {
        case FA_OK: return "ok";
        case FA_ERR_NULL: return "a required pointer is NULL";
        case FA_ERR_SHAPE: return "invalid or too large tensor shape";
        case FA_ERR_HEADDIM: return "unsupported head dimension (forward: 64, 128, 256, 512, 1024; decode and backward: 64, 128)";
        case FA_ERR_DTYPE: return "dtype must be FA_FP16 or FA_BF16";
        case FA_ERR_ALIGN: return "tensor pointer is not 16-byte aligned";
        case FA_ERR_SPLITS: return "num_splits must be in [1, min(Sk, FA_MAX_SPLITS)]";
        case FA_ERR_SCALE: return "scale must be finite and positive";
        case FA_ERR_CUDA: return "CUDA runtime error";
        case FA_ERR_DEVICE_TIMEOUT: return "a kernel abandoned a barrier wait (device timeout)";
        case FA_ERR_SCRATCH: return "problem larger than the built-in decode scratch";
        case FA_ERR_DEVICE_INDEX: return "a kernel met an out-of-range block-table entry";
        case FA_ERR_WORKSPACE: return "workspace smaller than fa_bwd_workspace_bytes()";
        case FA_ERR_DEVICE_SEQLENS:
            return "cu_seqlens do not describe sequences inside total_q/total_k, or a query sequence is longer "
                   "than max_seqlen_q (nothing was computed)";
    }
    return "unknown status";
}

fa_status_t fa_fwd(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H, int Sq, int Sk,
                   int D, int causal, float scale, fa_dtype_t dtype, void *stream) {
    if (!q || !k || !v || !o || !lse) return FA_ERR_NULL;
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_DTYPE;
    if (!fwd_head_dim_ok(D)) return FA_ERR_HEADDIM;
    if (B < 1 || H < 1 || Sq < 1 || Sk < 1 || Sq > kMaxLen || Sk > kMaxLen) return FA_ERR_SHAPE;
    const long long BH = static_cast<long long>(B) * H;
    const long long n_pairs = ((Sq + 127) / 128 + 1) / 2;
    const long long n_work = fwd_work_items(D, BH, Sq);
    if (BH > INT_MAX || n_work > INT_MAX) return FA_ERR_SHAPE;
    if (!scale_ok(scale)) return FA_ERR_SCALE;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned4(lse)) return FA_ERR_ALIGN;

    const bool bf16 = dtype == FA_BF16;
    CUtensorMap maps[3];
    const uint64_t row = static_cast<uint64_t>(D) * 2;
    const uint32_t kv_rows = D >= 256 ? 64 : 128;  // K/V tile height of the kernel that runs
    if (!encode_map(&maps[0], bf16, q, D, Sq, BH, row, row * Sq, 128, 1) ||
        !encode_map(&maps[1], bf16, k, D, Sk, BH, row, row * Sk, kv_rows, 1) ||
        !encode_map(&maps[2], bf16, v, D, Sk, BH, row, row * Sk, kv_rows, 1))
        return FA_ERR_CUDA;
    int *err = device_error_word();
    const int sms = num_sms();
    if (err == nullptr || sms <= 0) return FA_ERR_CUDA;

    fa::FwdParams p{};
    p.o = o;
    p.lse = lse;
    p.B = B;
    p.H = H;
    p.Sq = Sq;
    p.Sk = Sk;
    p.total_q = 0;
    p.n_pairs = static_cast<int>(n_pairs);
    p.n_qtiles = (Sq + 127) / 128;
    p.num_work = static_cast<int>(n_work);
    p.scale_log2 = scale * kLog2e;
    p.err = err;
    p.timeout_ns = g_wait_limit_ns.load();
    p.withhold = g_withhold.load();
    const int grid = p.num_work < sms ? p.num_work : sms;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = D > 256    ? fa::launch_fwd_splitd(D, bf16, causal != 0, false, maps, p, grid, st)
                          : D == 256 ? fa::launch_fwd_d256(bf16, causal != 0, false, maps, p, grid, st)
                                     : fa::launch_fwd_dense(D, bf16, causal != 0, maps, p, grid, st);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_fwd_varlen(const void *q, const void *k, const void *v, void *o, float *lse,
                          const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int num_seqs, int total_q,
                          int total_k, int max_seqlen_q, int H, int D, int causal, float scale, fa_dtype_t dtype,
                          void *stream) {
    if (!q || !k || !v || !o || !lse || !cu_seqlens_q || !cu_seqlens_k) return FA_ERR_NULL;
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_DTYPE;
    if (!fwd_head_dim_ok(D)) return FA_ERR_HEADDIM;
    if (num_seqs < 1 || total_q < 1 || total_k < 1 || max_seqlen_q < 1 || H < 1 || max_seqlen_q > kMaxLen ||
        total_q > kMaxLen || total_k > kMaxLen)
        return FA_ERR_SHAPE;
    const long long SH = static_cast<long long>(num_seqs) * H;
    const long long n_pairs = ((max_seqlen_q + 127) / 128 + 1) / 2;
    const long long n_work = fwd_work_items(D, SH, max_seqlen_q);
    if (SH > INT_MAX || n_work > INT_MAX) return FA_ERR_SHAPE;
    if (!scale_ok(scale)) return FA_ERR_SCALE;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned4(lse)) return FA_ERR_ALIGN;

    const bool bf16 = dtype == FA_BF16;
    CUtensorMap maps[3];
    const uint64_t row = static_cast<uint64_t>(D) * 2;
    const uint64_t tok = row * H;
    const uint32_t kv_rows = D >= 256 ? 64 : 128;
    if (!encode_map(&maps[0], bf16, q, D, H, total_q, row, tok, 1, 128) ||
        !encode_map(&maps[1], bf16, k, D, H, total_k, row, tok, 1, kv_rows) ||
        !encode_map(&maps[2], bf16, v, D, H, total_k, row, tok, 1, kv_rows))
        return FA_ERR_CUDA;
    int *err = device_error_word();
    const int sms = num_sms();
    if (err == nullptr || sms <= 0) return FA_ERR_CUDA;

    fa::FwdParams p{};
    p.o = o;
    p.lse = lse;
    p.cu_q = cu_seqlens_q;
    p.cu_k = cu_seqlens_k;
    p.B = num_seqs;
    p.H = H;
    p.Sq = max_seqlen_q;
    p.Sk = 0;
    p.total_q = total_q;
    p.total_k = total_k;
    p.n_pairs = static_cast<int>(n_pairs);
    p.n_qtiles = (max_seqlen_q + 127) / 128;
    p.num_work = static_cast<int>(n_work);
    p.scale_log2 = scale * kLog2e;
    p.err = err;
    p.timeout_ns = g_wait_limit_ns.load();
    p.withhold = g_withhold.load();
    const int grid = p.num_work < sms ? p.num_work : sms;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = D > 256    ? fa::launch_fwd_splitd(D, bf16, causal != 0, true, maps, p, grid, st)
                          : D == 256 ? fa::launch_fwd_d256(bf16, causal != 0, true, maps, p, grid, st)
                                     : fa::launch_fwd_varlen(D, bf16, causal != 0, maps, p, grid, st);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_decode_splitkv(const void *q, const void *k, const void *v, float *o_part, float *m_part,
                              float *l_part, int B, int H, int Sk, int D, int num_splits, float scale,
                              fa_dtype_t dtype, void *stream) {
    if (!q || !k || !v || !o_part || !m_part || !l_part) return FA_ERR_NULL;
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_DTYPE;
    if (D != 64 && D != 128) return FA_ERR_HEADDIM;
    if (B < 1 || H < 1 || Sk < 1 || Sk > kMaxLen) return FA_ERR_SHAPE;
    if (num_splits < 1 || num_splits > Sk || num_splits > FA_MAX_SPLITS) return FA_ERR_SPLITS;
    const long long BH = static_cast<long long>(B) * H;
    if (BH * num_splits > INT_MAX) return FA_ERR_SHAPE;
    if (!scale_ok(scale)) return FA_ERR_SCALE;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned4(o_part) || !aligned4(m_part) ||
        !aligned4(l_part))
        return FA_ERR_ALIGN;
    const int P = (Sk + num_splits - 1) / num_splits;
    const cudaError_t e = fa::launch_decode_split(D, dtype == FA_BF16, q, k, v, o_part, m_part, l_part,
                                                  static_cast<int>(BH), Sk, num_splits, P, scale * kLog2e,
                                                  static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_decode_paged_splitkv(const void *q, const void *k_cache, const void *v_cache,
                                    const int32_t *block_table, const int32_t *seq_lens, float *o_part,
                                    float *m_part, float *l_part, int B, int H, int D, int num_blocks,
                                    int block_size, int max_blocks_per_seq, int num_splits, float scale,
                                    fa_dtype_t dtype, void *stream) {
    if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !o_part || !m_part || !l_part)
        return FA_ERR_NULL;
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_DTYPE;
    if (D != 64 && D != 128) return FA_ERR_HEADDIM;
    if (B < 1 || H < 1 || num_blocks < 1 || max_blocks_per_seq < 1) return FA_ERR_SHAPE;
    if (block_size < 1 || block_size > 1024 || (block_size & (block_size - 1)) != 0) return FA_ERR_SHAPE;
    if (static_cast<long long>(max_blocks_per_seq) * block_size > kMaxLen) return FA_ERR_SHAPE;
    if (num_splits < 1 || num_splits > FA_MAX_SPLITS) return FA_ERR_SPLITS;
    const long long BH = static_cast<long long>(B) * H;
    if (BH * num_splits > INT_MAX || static_cast<long long>(num_blocks) * H > INT_MAX) return FA_ERR_SHAPE;
    if (!scale_ok(scale)) return FA_ERR_SCALE;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned4(block_table) ||
        !aligned4(seq_lens) || !aligned4(o_part) || !aligned4(m_part) || !aligned4(l_part))
        return FA_ERR_ALIGN;
    int *err = device_error_word();
    if (err == nullptr) return FA_ERR_CUDA;
    int log2_bs = 0;
    while ((1 << log2_bs) < block_size) ++log2_bs;
    fa::DecodeParams p{};
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k_cache);
    p.v = static_cast<const uint16_t *>(v_cache);
    p.o_part = o_part;
    p.m_part = m_part;
    p.l_part = l_part;
    p.H = H;
    p.num_splits = num_splits;
    p.scale_log2 = scale * kLog2e;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.max_blocks = max_blocks_per_seq;
    p.log2_bs = log2_bs;
    p.num_blocks = num_blocks;
    p.err = err;
    const cudaError_t e =
        fa::launch_decode_split_paged(D, dtype == FA_BF16, p, static_cast<int>(BH), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_decode_splitkv_fused(const void *q, const void *k, const void *v, void *o, float *lse, float *o_part,
                                    float *m_part, float *l_part, int32_t *counters, int B, int H, int Sk, int D,
                                    int num_splits, float scale, fa_dtype_t dtype, void *stream) {
    if (!q || !k || !v || !o || !lse || !o_part || !m_part || !l_part || !counters) return FA_ERR_NULL;
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_DTYPE;
    if (D != 64 && D != 128) return FA_ERR_HEADDIM;
    if (B < 1 || H < 1 || Sk < 1 || Sk > kMaxLen) return FA_ERR_SHAPE;
    if (num_splits < 1 || num_splits > Sk || num_splits > FA_MAX_SPLITS) return FA_ERR_SPLITS;
    const long long BH = static_cast<long long>(B) * H;
    if (BH * num_splits > INT_MAX) return FA_ERR_SHAPE;
    if (!scale_ok(scale)) return FA_ERR_SCALE;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned4(lse) || !aligned4(o_part) ||
        !aligned4(m_part) || !aligned4(l_part) || !aligned4(counters))
        return FA_ERR_ALIGN;
    fa::DecodeParams p{};
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.o_part = o_part;
    p.m_part = m_part;
    p.l_part = l_part;
    p.H = H;
    p.Sk = Sk;
    p.num_splits = num_splits;
    p.keys_per_split = (Sk + num_splits - 1) / num_splits;
    p.scale_log2 = scale * kLog2e;
    p.o = o;
    p.lse = lse;
    p.counters = counters;
    const cudaError_t e = fa::launch_decode_fused(D, dtype == FA_BF16, false, p, static_cast<int>(BH),
                                                  static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_decode_paged_splitkv_fused(const void *q, const void *k_cache, const void *v_cache,
                                          const int32_t *block_table, const int32_t *seq_lens, void *o, float *lse,
                                          float *o_part, float *m_part, float *l_part, int32_t *counters, int B,
                                          int H, int D, int num_blocks, int block_size, int max_blocks_per_seq,
                                          int num_splits, float scale, fa_dtype_t dtype, void *stream) {
    if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !o || !lse || !o_part || !m_part || !l_part ||
        !counters)
        return FA_ERR_NULL;
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_DTYPE;
    if (D != 64 && D != 128) return FA_ERR_HEADDIM;
    if (B < 1 || H < 1 || num_blocks < 1 || max_blocks_per_seq < 1) return FA_ERR_SHAPE;
    if (block_size < 1 || block_size > 1024 || (block_size & (block_size - 1)) != 0) return FA_ERR_SHAPE;
    if (static_cast<long long>(max_blocks_per_seq) * block_size > kMaxLen) return FA_ERR_SHAPE;
    if (num_splits < 1 || num_splits > FA_MAX_SPLITS) return FA_ERR_SPLITS;
    const long long BH = static_cast<long long>(B) * H;
    if (BH * num_splits > INT_MAX || static_cast<long long>(num_blocks) * H > INT_MAX) return FA_ERR_SHAPE;
    if (!scale_ok(scale)) return FA_ERR_SCALE;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned4(block_table) ||
        !aligned4(seq_lens) || !aligned16(o) || !aligned4(lse) || !aligned4(o_part) || !aligned4(m_part) ||
        !aligned4(l_part) || !aligned4(counters))
        return FA_ERR_ALIGN;
    int *err = device_error_word();
    if (err == nullptr) return FA_ERR_CUDA;
    int log2_bs = 0;
    while ((1 << log2_bs) < block_size) ++log2_bs;
    fa::DecodeParams p{};
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k_cache);
    p.v = static_cast<const uint16_t *>(v_cache);
    p.o_part = o_part;
    p.m_part = m_part;
    p.l_part = l_part;
    p.H = H;
    p.num_splits = num_splits;
    p.scale_log2 = scale * kLog2e;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.max_blocks = max_blocks_per_seq;
    p.log2_bs = log2_bs;
    p.num_blocks = num_blocks;
    p.err = err;
    p.o = o;
    p.lse = lse;
    p.counters = counters;
    const cudaError_t e = fa::launch_decode_fused(D, dtype == FA_BF16, true, p, static_cast<int>(BH),
                                                  static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_bwd_workspace_bytes(int B, int H, int Sq, int D) {
    if (B < 1 || H < 1 || Sq < 1 || Sq > kMaxLen || (D != 64 && D != 128)) return 0;
    const long long BH = static_cast<long long>(B) * H;
    if (BH > INT_MAX) return 0;
    const long long pad = (static_cast<long long>(Sq) + 127) / 128 * 128;
    // + 16 bytes: the main kernel's work counter
    return static_cast<size_t>(BH * Sq * D + 2 * BH * pad) * sizeof(float) + 16;
}

fa_status_t fa_bwd(const void *q, const void *k, const void *v, const void *o, const void *dout, const float *lse,
                   void *dq, void *dk, void *dv, float *workspace, size_t workspace_bytes, int B, int H, int Sq,
                   int Sk, int D, int causal, float scale, fa_dtype_t dtype, void *stream) {
    if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv || !workspace) return FA_ERR_NULL;
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_DTYPE;
    if (D != 64 && D != 128) return FA_ERR_HEADDIM;
    if (B < 1 || H < 1 || Sq < 1 || Sk < 1 || Sq > kMaxLen || Sk > kMaxLen) return FA_ERR_SHAPE;
    const long long BH = static_cast<long long>(B) * H;
    const long long n_kt = (Sk + 127) / 128;
    if (BH > INT_MAX || BH * n_kt > INT_MAX) return FA_ERR_SHAPE;
    if (!scale_ok(scale)) return FA_ERR_SCALE;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) || !aligned4(lse) ||
        !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(workspace))
        return FA_ERR_ALIGN;
    const size_t need = fa_bwd_workspace_bytes(B, H, Sq, D);
    if (need == 0) return FA_ERR_SHAPE;
    if (workspace_bytes < need) return FA_ERR_WORKSPACE;

    const bool bf16 = dtype == FA_BF16;
    CUtensorMap maps[5];
    const uint64_t row = static_cast<uint64_t>(D) * 2;
    const uint32_t q_rows = D == 128 ? 64 : 128;  // query rows per step of the kernel that runs
    if (!encode_map(&maps[0], bf16, q, D, Sq, BH, row, row * Sq, q_rows, 1) ||
        !encode_map(&maps[1], bf16, k, D, Sk, BH, row, row * Sk, 128, 1) ||
        !encode_map(&maps[2], bf16, v, D, Sk, BH, row, row * Sk, 128, 1) ||
        !encode_map(&maps[3], bf16, dout, D, Sq, BH, row, row * Sq, q_rows, 1) ||
        !encode_map_f32(&maps[4], workspace, D, Sq, BH, D * 4, D * 4 * static_cast<uint64_t>(Sq), q_rows, 1))
        return FA_ERR_CUDA;
    int *err = device_error_word();
    if (err == nullptr) return FA_ERR_CUDA;

    fa::BwdParams p{};
    p.BH = static_cast<int>(BH);
    p.Sq = Sq;
    p.Sk = Sk;
    p.n_qtiles = (Sq + 127) / 128;
    p.n_ktiles = static_cast<int>(n_kt);
    p.Sq_pad = p.n_qtiles * 128;
    p.heads_per_group = bwd_units_per_group(BH, Sq, D);
    p.dq_acc = workspace;
    p.lse2 = workspace + static_cast<size_t>(BH) * Sq * D;
    p.delta = p.lse2 + static_cast<size_t>(BH) * p.Sq_pad;
    p.work_counter = reinterpret_cast<int *>(p.delta + static_cast<size_t>(BH) * p.Sq_pad);
    p.total_units = static_cast<int>(BH * n_kt);
    p.grid = num_sms();
    if (p.grid <= 0) return FA_ERR_CUDA;
    p.dk = dk;
    p.dv = dv;
    p.scale = scale;
    p.scale_log2 = scale * kLog2e;
    p.err = err;
    p.timeout_ns = g_wait_limit_ns.load();
    p.withhold = g_withhold.load();
    const cudaError_t e = fa::launch_bwd_dense(D, bf16, causal != 0, maps, o, dout, lse, dq, p,
                                         static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_bwd_varlen_workspace_bytes(int total_q, int H, int D) {
    if (total_q < 1 || H < 1 || total_q > kMaxLen || (D != 64 && D != 128)) return 0;
    const long long TH = static_cast<long long>(total_q) * H;
    if (TH > INT_MAX) return 0;
    return static_cast<size_t>(TH * D + 2 * TH) * sizeof(float) + 16;  // + the work counter
}

fa_status_t fa_bwd_varlen(const void *q, const void *k, const void *v, const void *o, const void *dout,
                          const float *lse, void *dq, void *dk, void *dv, float *workspace, size_t workspace_bytes,
                          const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int num_seqs, int total_q,
                          int total_k, int max_seqlen_q, int max_seqlen_k, int H, int D, int causal, float scale,
                          fa_dtype_t dtype, void *stream) {
    if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv || !workspace || !cu_seqlens_q || !cu_seqlens_k)
        return FA_ERR_NULL;
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_DTYPE;
    if (D != 64 && D != 128) return FA_ERR_HEADDIM;
    if (num_seqs < 1 || total_q < 1 || total_k < 1 || max_seqlen_q < 1 || max_seqlen_k < 1 || H < 1 ||
        total_q > kMaxLen || total_k > kMaxLen || max_seqlen_q > kMaxLen || max_seqlen_k > kMaxLen)
        return FA_ERR_SHAPE;
    const long long units = static_cast<long long>(num_seqs) * H;
    const long long n_kt = (max_seqlen_k + 127) / 128;
    if (units > INT_MAX || units * n_kt > INT_MAX || static_cast<long long>(total_q) * H > INT_MAX ||
        static_cast<long long>(total_k) * H > INT_MAX)
        return FA_ERR_SHAPE;
    if (!scale_ok(scale)) return FA_ERR_SCALE;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) || !aligned4(lse) ||
        !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(workspace) || !aligned4(cu_seqlens_q) ||
        !aligned4(cu_seqlens_k))
        return FA_ERR_ALIGN;
    const size_t need = fa_bwd_varlen_workspace_bytes(total_q, H, D);
    if (need == 0) return FA_ERR_SHAPE;
    if (workspace_bytes < need) return FA_ERR_WORKSPACE;

    const bool bf16 = dtype == FA_BF16;
    CUtensorMap maps[5];
    const uint64_t row = static_cast<uint64_t>(D) * 2;
    const uint64_t tok = row * H;
    const uint32_t q_rows = D == 128 ? 64 : 128;  // query rows per step of the kernel that runs
    if (!encode_map(&maps[0], bf16, q, D, H, total_q, row, tok, 1, q_rows) ||
        !encode_map(&maps[1], bf16, k, D, H, total_k, row, tok, 1, 128) ||
        !encode_map(&maps[2], bf16, v, D, H, total_k, row, tok, 1, 128) ||
        !encode_map(&maps[3], bf16, dout, D, H, total_q, row, tok, 1, q_rows) ||
        !encode_map_f32(&maps[4], workspace, D, H, total_q, D * 4, D * 4 * static_cast<uint64_t>(H), 1, q_rows))
        return FA_ERR_CUDA;
    int *err = device_error_word();
    if (err == nullptr) return FA_ERR_CUDA;

    fa::BwdParams p{};
    p.BH = static_cast<int>(units);
    p.Sq = max_seqlen_q;
    p.Sk = max_seqlen_k;
    p.n_qtiles = (max_seqlen_q + 127) / 128;
    p.n_ktiles = static_cast<int>(n_kt);
    p.Sq_pad = 0;
    p.heads_per_group = bwd_units_per_group(units, max_seqlen_q, D);
    p.cu_q = cu_seqlens_q;
    p.cu_k = cu_seqlens_k;
    p.H = H;
    p.total_q = total_q;
    p.total_k = total_k;
    p.dq_acc = workspace;
    p.lse2 = workspace + static_cast<size_t>(total_q) * H * D;
    p.delta = p.lse2 + static_cast<size_t>(total_q) * H;
    p.work_counter = reinterpret_cast<int *>(p.delta + static_cast<size_t>(total_q) * H);
    p.total_units = p.BH * p.n_ktiles;
    p.grid = num_sms();
    if (p.grid <= 0) return FA_ERR_CUDA;
    p.dk = dk;
    p.dv = dv;
    p.scale = scale;
    p.scale_log2 = scale * kLog2e;
    p.err = err;
    p.timeout_ns = g_wait_limit_ns.load();
    p.withhold = g_withhold.load();
    const cudaError_t e = fa::launch_bwd_varlen(D, bf16, causal != 0, maps, o, dout, lse, dq, p,
                                                static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_splitkv_merge(const float *o_part, const float *m_part, const float *l_part, void *o, float *lse,
                             int B, int H, int D, int num_splits, fa_dtype_t dtype, void *stream) {
    if (!o_part || !m_part || !l_part || !o || !lse) return FA_ERR_NULL;
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_DTYPE;
    if (D != 64 && D != 128) return FA_ERR_HEADDIM;
    if (B < 1 || H < 1) return FA_ERR_SHAPE;
    if (num_splits < 1 || num_splits > FA_MAX_SPLITS) return FA_ERR_SPLITS;
    const long long BH = static_cast<long long>(B) * H;
    if (BH > INT_MAX) return FA_ERR_SHAPE;
    if (!aligned4(o_part) || !aligned4(m_part) || !aligned4(l_part) || !aligned16(o) || !aligned4(lse))
        return FA_ERR_ALIGN;
    const cudaError_t e = fa::launch_splitkv_merge(D, dtype == FA_BF16, o_part, m_part, l_part, o, lse,
                                                   static_cast<int>(BH), num_splits,
                                                   static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// Sliding-window attention, dense (cu_q == nullptr: B sequences of Sq queries
// and Sk keys) or packed (B sequences, at most Sq queries and Sk keys each).
static bool window_ok(int H, int Hkv, int Sq, int Sk, int window, int sinks) {
    return H >= 1 && Hkv >= 1 && H % Hkv == 0 && Sq >= 1 && Sk >= 1 && Sq <= kMaxWindowLen && Sk <= kMaxWindowLen &&
           window >= 1 && sinks >= 0;
}

static fa_status_t fwd_window(const void *q, const void *k, const void *v, void *o, float *lse,
                              const int32_t *cu_q, const int32_t *cu_k, int B, int total_q, int total_k, int H,
                              int Hkv, int Sq, int Sk, int D, int window, int sinks, float scale, fa_dtype_t dtype,
                              void *stream) {
    const bool varlen = cu_q != nullptr;
    const long long SH = static_cast<long long>(B) * H;
    const long long n_work = fwd_work_items(D, SH, Sq);
    if (SH > INT_MAX || n_work > INT_MAX) return FA_ERR_SHAPE;
    if (!scale_ok(scale)) return FA_ERR_SCALE;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned4(lse) || !aligned4(cu_q) ||
        !aligned4(cu_k))
        return FA_ERR_ALIGN;

    const bool bf16 = dtype == FA_BF16;
    CUtensorMap maps[3];
    const uint64_t row = static_cast<uint64_t>(D) * 2;
    const bool maps_ok =
        varlen ? encode_map(&maps[0], bf16, q, D, H, total_q, row, row * H, 1, 128) &&
                     encode_map(&maps[1], bf16, k, D, Hkv, total_k, row, row * Hkv, 1, 128) &&
                     encode_map(&maps[2], bf16, v, D, Hkv, total_k, row, row * Hkv, 1, 128)
               : encode_map(&maps[0], bf16, q, D, Sq, SH, row, row * Sq, 128, 1) &&
                     encode_map(&maps[1], bf16, k, D, Sk, SH / H * Hkv, row, row * Sk, 128, 1) &&
                     encode_map(&maps[2], bf16, v, D, Sk, SH / H * Hkv, row, row * Sk, 128, 1);
    int *err = device_error_word();
    const int sms = num_sms();
    if (!maps_ok || err == nullptr || sms <= 0) return FA_ERR_CUDA;

    fa::FwdParams p{};
    p.o = o;
    p.lse = lse;
    p.cu_q = cu_q;
    p.cu_k = cu_k;
    p.B = B;
    p.H = H;
    p.Sq = Sq;
    p.Sk = Sk;
    p.total_q = total_q;
    p.total_k = total_k;
    p.n_qtiles = (Sq + 127) / 128;
    p.n_pairs = (p.n_qtiles + 1) / 2;
    p.num_work = static_cast<int>(n_work);
    p.scale_log2 = scale * kLog2e;
    p.err = err;
    p.timeout_ns = g_wait_limit_ns.load();
    p.withhold = g_withhold.load();
    p.window = window < kMaxWindowLen ? window : kMaxWindowLen;
    p.sinks = sinks < kMaxWindowLen ? sinks : kMaxWindowLen;
    p.group = H / Hkv;
    const int grid = p.num_work < sms ? p.num_work : sms;
    const cudaError_t e =
        fa::launch_fwd_window(D, bf16, varlen, maps, p, grid, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_fwd_window(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H, int Hkv,
                          int Sq, int Sk, int D, int window, int sinks, float scale, fa_dtype_t dtype, void *stream) {
    if (!q || !k || !v || !o || !lse) return FA_ERR_NULL;
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_DTYPE;
    if (D != 64 && D != 128) return FA_ERR_HEADDIM;
    if (B < 1 || !window_ok(H, Hkv, Sq, Sk, window, sinks)) return FA_ERR_SHAPE;
    return fwd_window(q, k, v, o, lse, nullptr, nullptr, B, 0, 0, H, Hkv, Sq, Sk, D, window, sinks, scale, dtype,
                      stream);
}

fa_status_t fa_fwd_window_varlen(const void *q, const void *k, const void *v, void *o, float *lse,
                                 const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int num_seqs, int total_q,
                                 int total_k, int max_seqlen_q, int H, int Hkv, int D, int window, int sinks,
                                 float scale, fa_dtype_t dtype, void *stream) {
    if (!q || !k || !v || !o || !lse || !cu_seqlens_q || !cu_seqlens_k) return FA_ERR_NULL;
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_DTYPE;
    if (D != 64 && D != 128) return FA_ERR_HEADDIM;
    if (num_seqs < 1 || total_q < 1 || total_q > kMaxWindowLen ||
        !window_ok(H, Hkv, max_seqlen_q, total_k, window, sinks))
        return FA_ERR_SHAPE;
    return fwd_window(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k, H, Hkv, max_seqlen_q,
                      0, D, window, sinks, scale, dtype, stream);
}

// How the window backward cuts its key tiles' steps into segments, and the
// workspace that takes: fa_bwd's (base bytes) and the segments' dV and dK.
struct WindowCut {
    int sink_tiles, segs_sink, segs;
    size_t bytes;
};

static WindowCut window_cut(size_t base, long long units, int H, int Hkv, int Sq, int Sk, int D, int window,
                            int sinks) {
    WindowCut c{};
    const long long n_kt = (Sk + 127) / 128, block = D == 64 ? 128 : 64, group = H / Hkv;
    const long long sink_tiles = (static_cast<long long>(sinks) + 127) / 128;
    c.sink_tiles = static_cast<int>(sink_tiles < n_kt ? sink_tiles : n_kt);
    // steps of the longest plain tile and of the longest tile with sinks, in
    // the longest sequence
    const long long reach = 128LL + window < Sq ? 128LL + window : Sq;
    const long long plain = group * ((reach + block - 1) / block), sunk = group * ((Sq + block - 1) / block);
    // Plain tiles: the count of segments (up to 6, 1024 units in all) that makes
    // the launch shortest, in half steps: waves of units, each as long as its
    // steps and 3 to start and end; joining costs one for 64 columns and segment.
    // A wave takes some units more than there are SMs: the last ones are light.
    // (16 on 2 heads, 4 x 777 tokens, D = 128, window 200: 84, 56, 47, 56 us with 1 to
    // 4 segments, 3 taken; 6 on 2 heads, 2 x 777, D = 64, window 300: 35, 25, 21,
    // 18.5, 4 taken; 8 on 8 heads, 2048, D = 128, window 512: 29, 39, 43, 1 taken.)
    constexpr long long kSms = 152, kWave = 170;
    const long long tiles = units * n_kt;
    long long segs = 1, best = 0;
    for (long long n = 1; n <= 6 && (n == 1 || tiles * n <= 1024); ++n) {
        const long long waves = (tiles * n + kWave - 1) / kWave, steps = (plain + n - 1) / n + 3;
        const long long cost = 2 * waves * steps + (n > 1 ? n * (D / 64) : 0);
        if (n == 1 || cost < best) {
            best = cost;
            segs = n;
        }
    }
    // Tiles with sinks: no longer than the plain ones, or a quarter of an SM's
    // share where that is more.
    const long long others = units * (n_kt - c.sink_tiles);
    const long long share = (others * plain + units * c.sink_tiles * sunk) / (4 * kSms);
    const long long most = others > 0 && plain / segs > share ? plain / segs : (share > 8 ? share : 8);
    long long segs_sink = c.sink_tiles > 0 ? (sunk + most - 1) / most : 1;
    segs_sink = segs_sink < 1 ? 1 : (segs_sink < 64 ? segs_sink : 64);
    c.segs = static_cast<int>(segs);
    c.segs_sink = static_cast<int>(segs_sink);
    const long long slots = units * ((segs_sink > 1 ? c.sink_tiles * segs_sink : 0) +
                                     (segs > 1 ? (n_kt - c.sink_tiles) * segs : 0));
    c.bytes = (base + 15) / 16 * 16 + static_cast<size_t>(slots) * 2 * 128 * D * sizeof(float);
    return c;
}

size_t fa_bwd_window_workspace_bytes(int B, int H, int Hkv, int Sq, int Sk, int D, int window, int sinks) {
    if (B < 1 || !window_ok(H, Hkv, Sq, Sk, window, sinks)) return 0;
    const size_t base = fa_bwd_workspace_bytes(B, H, Sq, D);
    if (base == 0) return 0;
    return window_cut(base, static_cast<long long>(B) * Hkv, H, Hkv, Sq, Sk, D, window, sinks).bytes;
}

size_t fa_bwd_window_varlen_workspace_bytes(int num_seqs, int total_q, int max_seqlen_q, int max_seqlen_k, int H,
                                            int Hkv, int D, int window, int sinks) {
    if (num_seqs < 1 || !window_ok(H, Hkv, max_seqlen_q, max_seqlen_k, window, sinks)) return 0;
    const size_t base = fa_bwd_varlen_workspace_bytes(total_q, H, D);
    if (base == 0) return 0;
    return window_cut(base, static_cast<long long>(num_seqs) * Hkv, H, Hkv, max_seqlen_q, max_seqlen_k, D, window,
                      sinks).bytes;
}

static fa_status_t bwd_window(const void *q, const void *k, const void *v, const void *o, const void *dout,
                              const float *lse, void *dq, void *dk, void *dv, float *workspace,
                              size_t workspace_bytes, const int32_t *cu_q, const int32_t *cu_k, int B, int total_q,
                              int total_k, int H, int Hkv, int Sq, int Sk, int D, int window, int sinks, float scale,
                              fa_dtype_t dtype, void *stream) {
    const bool varlen = cu_q != nullptr;
    const long long BH = static_cast<long long>(B) * H, units = static_cast<long long>(B) * Hkv;
    const long long n_kt = (Sk + 127) / 128;
    if (BH > INT_MAX || units * n_kt > INT_MAX || static_cast<long long>(total_q) * H > INT_MAX ||
        static_cast<long long>(total_k) * Hkv > INT_MAX)
        return FA_ERR_SHAPE;
    if (!scale_ok(scale)) return FA_ERR_SCALE;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) || !aligned4(lse) ||
        !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(workspace) || !aligned4(cu_q) ||
        !aligned4(cu_k))
        return FA_ERR_ALIGN;
    const size_t base = varlen ? fa_bwd_varlen_workspace_bytes(total_q, H, D) : fa_bwd_workspace_bytes(B, H, Sq, D);
    if (base == 0) return FA_ERR_SHAPE;
    const WindowCut cut = window_cut(base, units, H, Hkv, Sq, Sk, D, window, sinks);
    const long long per_head = static_cast<long long>(cut.sink_tiles) * cut.segs_sink +
                               (n_kt - cut.sink_tiles) * cut.segs;
    if (units * per_head > INT_MAX) return FA_ERR_SHAPE;
    if (workspace_bytes < cut.bytes) return FA_ERR_WORKSPACE;

    const bool bf16 = dtype == FA_BF16;
    CUtensorMap maps[5];
    const uint64_t row = static_cast<uint64_t>(D) * 2, row4 = row * 2;
    const uint32_t q_rows = D == 128 ? 64 : 128;  // query rows per step of the kernel that runs
    const bool maps_ok =
        varlen ? encode_map(&maps[0], bf16, q, D, H, total_q, row, row * H, 1, q_rows) &&
                     encode_map(&maps[1], bf16, k, D, Hkv, total_k, row, row * Hkv, 1, 128) &&
                     encode_map(&maps[2], bf16, v, D, Hkv, total_k, row, row * Hkv, 1, 128) &&
                     encode_map(&maps[3], bf16, dout, D, H, total_q, row, row * H, 1, q_rows) &&
                     encode_map_f32(&maps[4], workspace, D, H, total_q, row4, row4 * H, 1, q_rows)
               : encode_map(&maps[0], bf16, q, D, Sq, BH, row, row * Sq, q_rows, 1) &&
                     encode_map(&maps[1], bf16, k, D, Sk, units, row, row * Sk, 128, 1) &&
                     encode_map(&maps[2], bf16, v, D, Sk, units, row, row * Sk, 128, 1) &&
                     encode_map(&maps[3], bf16, dout, D, Sq, BH, row, row * Sq, q_rows, 1) &&
                     encode_map_f32(&maps[4], workspace, D, Sq, BH, row4, row4 * Sq, q_rows, 1);
    int *err = device_error_word();
    const int sms = num_sms();
    if (!maps_ok || err == nullptr || sms <= 0) return FA_ERR_CUDA;

    fa::BwdParams p{};
    p.BH = static_cast<int>(BH);
    p.units = static_cast<int>(units);
    p.group = H / Hkv;
    p.Sq = Sq;
    p.Sk = Sk;
    p.n_qtiles = (Sq + 127) / 128;
    p.n_ktiles = static_cast<int>(n_kt);
    p.Sq_pad = varlen ? 0 : p.n_qtiles * 128;
    p.heads_per_group = bwd_units_per_group(units, static_cast<long long>(Sq) * p.group, D);
    p.cu_q = cu_q;
    p.cu_k = cu_k;
    p.H = H;
    p.total_q = total_q;
    p.total_k = total_k;
    const size_t rows = varlen ? static_cast<size_t>(total_q) * H : static_cast<size_t>(BH) * Sq;
    const size_t stat_rows = varlen ? rows : static_cast<size_t>(BH) * p.Sq_pad;
    p.dq_acc = workspace;
    p.lse2 = workspace + rows * D;
    p.delta = p.lse2 + stat_rows;
    p.work_counter = reinterpret_cast<int *>(p.delta + stat_rows);
    p.total_units = static_cast<int>(units * per_head);
    p.sink_tiles = cut.sink_tiles;
    p.segs_sink = cut.segs_sink;
    p.segs = cut.segs;
    p.segments = workspace + (base + 15) / 16 * 4;
    p.grid = sms;
    p.dk = dk;
    p.dv = dv;
    p.scale = scale;
    p.scale_log2 = scale * kLog2e;
    p.err = err;
    p.timeout_ns = g_wait_limit_ns.load();
    p.withhold = g_withhold.load();
    p.window = window < kMaxWindowLen ? window : kMaxWindowLen;
    p.sinks = sinks < kMaxWindowLen ? sinks : kMaxWindowLen;
    const cudaError_t e = fa::launch_bwd_window(D, bf16, varlen, maps, o, dout, lse, dq, p,
                                                static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_bwd_window(const void *q, const void *k, const void *v, const void *o, const void *dout,
                          const float *lse, void *dq, void *dk, void *dv, float *workspace, size_t workspace_bytes,
                          int B, int H, int Hkv, int Sq, int Sk, int D, int window, int sinks, float scale,
                          fa_dtype_t dtype, void *stream) {
    if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv || !workspace) return FA_ERR_NULL;
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_DTYPE;
    if (D != 64 && D != 128) return FA_ERR_HEADDIM;
    if (B < 1 || !window_ok(H, Hkv, Sq, Sk, window, sinks)) return FA_ERR_SHAPE;
    return bwd_window(q, k, v, o, dout, lse, dq, dk, dv, workspace, workspace_bytes, nullptr, nullptr, B, 0, 0, H,
                      Hkv, Sq, Sk, D, window, sinks, scale, dtype, stream);
}

fa_status_t fa_bwd_window_varlen(const void *q, const void *k, const void *v, const void *o, const void *dout,
                                 const float *lse, void *dq, void *dk, void *dv, float *workspace,
                                 size_t workspace_bytes, const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                 int num_seqs, int total_q, int total_k, int max_seqlen_q, int max_seqlen_k, int H,
                                 int Hkv, int D, int window, int sinks, float scale, fa_dtype_t dtype,
                                 void *stream) {
    if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv || !workspace || !cu_seqlens_q || !cu_seqlens_k)
        return FA_ERR_NULL;
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_DTYPE;
    if (D != 64 && D != 128) return FA_ERR_HEADDIM;
    if (num_seqs < 1 || total_q < 1 || total_k < 1 || total_q > kMaxWindowLen || total_k > kMaxWindowLen ||
        !window_ok(H, Hkv, max_seqlen_q, max_seqlen_k, window, sinks))
        return FA_ERR_SHAPE;
    return bwd_window(q, k, v, o, dout, lse, dq, dk, dv, workspace, workspace_bytes, cu_seqlens_q, cu_seqlens_k,
                      num_seqs, total_q, total_k, H, Hkv, max_seqlen_q, max_seqlen_k, D, window, sinks, scale, dtype,
                      stream);
}

static fa_status_t kv_q4(bool write, const void *k, const void *v, const void *k_codes, const void *k_scales,
                         const void *v_codes, const void *v_scales, const int32_t *block_table,
                         const int32_t *cu_seqlens, const int32_t *starts, int num_seqs, int total, int max_seqlen,
                         int Hkv, int D, int num_blocks, int block_size, int max_blocks_per_seq, fa_dtype_t dtype,
                         void *stream) {
    if (!k_codes || !k_scales || !v_codes || !v_scales || !block_table || !cu_seqlens) return FA_ERR_NULL;
    if ((!k || !v) && total != 0) return FA_ERR_NULL;
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_DTYPE;
    if (D != 64 && D != 128) return FA_ERR_HEADDIM;
    // (no tokens at all: the longest sequence may have none)
    if (num_seqs < 1 || total < 0 || total > kMaxLen || max_seqlen < (total > 0 ? 1 : 0) || max_seqlen > kMaxLen ||
        Hkv < 1)
        return FA_ERR_SHAPE;
    int log2_bs = 0;
    if (!pages_ok(Hkv, num_blocks, block_size, max_blocks_per_seq, log2_bs)) return FA_ERR_SHAPE;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_codes) || !aligned16(k_scales) || !aligned16(v_codes) ||
        !aligned16(v_scales) || !aligned4(block_table) || !aligned4(cu_seqlens) || !aligned4(starts))
        return FA_ERR_ALIGN;
    fa::KvQ4Params p{};
    p.k = const_cast<void *>(k);
    p.v = const_cast<void *>(v);
    p.k_codes = const_cast<void *>(k_codes);
    p.k_scales = const_cast<void *>(k_scales);
    p.v_codes = const_cast<void *>(v_codes);
    p.v_scales = const_cast<void *>(v_scales);
    p.block_table = block_table;
    p.cu_seqlens = cu_seqlens;
    p.starts = starts;
    p.total = total;
    p.max_seqlen = max_seqlen;
    p.Hkv = Hkv;
    p.num_blocks = num_blocks;
    p.log2_bs = log2_bs;
    p.max_blocks = max_blocks_per_seq;
    const long long grid = fa::kv_q4_grid(D, num_seqs, p);
    if (grid > INT_MAX) return FA_ERR_SHAPE;
    if (total == 0) return FA_OK;
    p.err = device_error_word();
    if (p.err == nullptr) return FA_ERR_CUDA;
    const cudaError_t e = fa::launch_kv_q4(D, dtype == FA_BF16, write, p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_kv_write_q4(const void *k, const void *v, void *k_codes, void *k_scales, void *v_codes, void *v_scales,
                           const int32_t *block_table, const int32_t *cu_seqlens, const int32_t *starts, int num_seqs,
                           int total, int max_seqlen, int Hkv, int D, int num_blocks, int block_size,
                           int max_blocks_per_seq, fa_dtype_t dtype, void *stream) {
    return kv_q4(true, k, v, k_codes, k_scales, v_codes, v_scales, block_table, cu_seqlens, starts, num_seqs, total,
                 max_seqlen, Hkv, D, num_blocks, block_size, max_blocks_per_seq, dtype, stream);
}

fa_status_t fa_kv_read_q4(void *k, void *v, const void *k_codes, const void *k_scales, const void *v_codes,
                          const void *v_scales, const int32_t *block_table, const int32_t *cu_seqlens,
                          const int32_t *starts, int num_seqs, int total, int max_seqlen, int Hkv, int D,
                          int num_blocks, int block_size, int max_blocks_per_seq, fa_dtype_t dtype, void *stream) {
    return kv_q4(false, k, v, k_codes, k_scales, v_codes, v_scales, block_table, cu_seqlens, starts, num_seqs, total,
                 max_seqlen, Hkv, D, num_blocks, block_size, max_blocks_per_seq, dtype, stream);
}

int fa_decode_splits(int B, int H, int Hkv, int max_keys) {
    if (B < 1 || H < 1 || Hkv < 1 || max_keys < 1) return 1;
    const int sms = num_sms();
    return fa::decode_gqa_splits(sms > 0 ? sms : 152, B, H, Hkv, max_keys);
}

static fa_status_t decode_gqa(bool q4, const void *q, const void *k, const void *ks, const void *v, const void *vs,
                              const int32_t *block_table, const int32_t *seq_lens, void *o, float *lse,
                              float *o_part, float *m_part, float *l_part, int32_t *counters, int B, int H, int Hkv,
                              int D, int num_blocks, int block_size, int max_blocks_per_seq, int num_splits,
                              int window, int sinks, float scale, fa_dtype_t dtype, void *stream) {
    if (!q || !k || !v || (q4 && (!ks || !vs)) || !block_table || !seq_lens || !o || !lse || !o_part || !m_part ||
        !l_part || !counters)
        return FA_ERR_NULL;
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_DTYPE;
    if (D != 64 && D != 128) return FA_ERR_HEADDIM;
    if (B < 1 || H < 1 || Hkv < 1 || H % Hkv != 0 || window < 0 || sinks < 0) return FA_ERR_SHAPE;
    int log2_bs = 0;
    if (!pages_ok(Hkv, num_blocks, block_size, max_blocks_per_seq, log2_bs)) return FA_ERR_SHAPE;
    // the 4-bit kernel counts rows in sixteens, in 32 bits (4 TB of codes)
    if (q4 && (static_cast<long long>(num_blocks) * Hkv << log2_bs) / 16 >= 0xffffffffLL) return FA_ERR_SHAPE;
    if (num_splits < 1 || num_splits > FA_MAX_SPLITS) return FA_ERR_SPLITS;
    if (static_cast<long long>(B) * H * num_splits > INT_MAX) return FA_ERR_SHAPE;
    if (!scale_ok(scale)) return FA_ERR_SCALE;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(ks) || !aligned16(vs) ||
        !aligned4(block_table) || !aligned4(seq_lens) || !aligned16(o) || !aligned4(lse) || !aligned16(o_part) ||
        !aligned4(m_part) || !aligned4(l_part) || !aligned4(counters))
        return FA_ERR_ALIGN;
    fa::GqaDecodeParams p{};
    p.q = static_cast<const uint16_t *>(q);
    p.k = k;
    p.v = v;
    p.ks = ks;
    p.vs = vs;
    p.o_part = o_part;
    p.m_part = m_part;
    p.l_part = l_part;
    p.o = o;
    p.lse = lse;
    p.counters = counters;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.H = H;
    p.Hkv = Hkv;
    p.group = H / Hkv;
    p.B = B;
    p.num_splits = num_splits;
    p.window = window;
    p.sinks = sinks;
    p.max_blocks = max_blocks_per_seq;
    p.log2_bs = log2_bs;
    p.num_blocks = num_blocks;
    p.scale_log2 = scale * kLog2e;
    p.err = device_error_word();
    const int sms = num_sms();
    if (p.err == nullptr || sms <= 0) return FA_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = q4 ? fa::launch_decode_q4(D, dtype == FA_BF16, p, sms, st)
                             : fa::launch_decode_window(D, dtype == FA_BF16, p, sms, st);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_decode_paged_window(const void *q, const void *k_cache, const void *v_cache,
                                   const int32_t *block_table, const int32_t *seq_lens, void *o, float *lse,
                                   float *o_part, float *m_part, float *l_part, int32_t *counters, int B, int H,
                                   int Hkv, int D, int num_blocks, int block_size, int max_blocks_per_seq,
                                   int num_splits, int window, int sinks, float scale, fa_dtype_t dtype,
                                   void *stream) {
    return decode_gqa(false, q, k_cache, nullptr, v_cache, nullptr, block_table, seq_lens, o, lse, o_part, m_part,
                      l_part, counters, B, H, Hkv, D, num_blocks, block_size, max_blocks_per_seq, num_splits, window,
                      sinks, scale, dtype, stream);
}

fa_status_t fa_decode_paged_q4(const void *q, const void *k_codes, const void *k_scales, const void *v_codes,
                               const void *v_scales, const int32_t *block_table, const int32_t *seq_lens, void *o,
                               float *lse, float *o_part, float *m_part, float *l_part, int32_t *counters, int B,
                               int H, int Hkv, int D, int num_blocks, int block_size, int max_blocks_per_seq,
                               int num_splits, int window, int sinks, float scale, fa_dtype_t dtype, void *stream) {
    return decode_gqa(true, q, k_codes, k_scales, v_codes, v_scales, block_table, seq_lens, o, lse, o_part, m_part,
                      l_part, counters, B, H, Hkv, D, num_blocks, block_size, max_blocks_per_seq, num_splits, window,
                      sinks, scale, dtype, stream);
}

fa_status_t fa_test_withhold_load(int load, unsigned long long wait_limit_ns) {
    if (load < 0) return FA_ERR_SHAPE;
    g_withhold.store(load);
    g_wait_limit_ns.store(wait_limit_ns == 0 ? fa::kWaitTimeoutNs : wait_limit_ns);
    return FA_OK;
}

fa_status_t fa_check_device_error(void *stream) {
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return FA_ERR_CUDA;
    int *err = device_error_word();
    if (err == nullptr) return FA_ERR_CUDA;
    int host = 0;
    if (cudaMemcpy(&host, err, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return FA_ERR_CUDA;
    if (host == 0) return FA_OK;
    const int zero = 0;
    if (cudaMemcpy(err, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess) return FA_ERR_CUDA;
    if (host == fa::kDeviceErrBadIndex) return FA_ERR_DEVICE_INDEX;
    if (host == fa::kDeviceErrSeqLens) return FA_ERR_DEVICE_SEQLENS;
    return FA_ERR_DEVICE_TIMEOUT;
}

}  // extern "C"
