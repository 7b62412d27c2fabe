// kq8_internal.h -- launchers shared between the libkq8 translation units.
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "kq8.h"
#include "kq8_common.cuh"

namespace kq8 {

struct AttnParams;
struct SparseParams;
struct PrefillParams;

// Largest element stride a call takes (a token or head index times it stays
// inside 64 bits).
constexpr size_t MAX_STRIDE = (size_t)1 << 31;
// Bytes from the first to the last element of n1 x n2 rows of HD elements at strides s1
// and s2 (in elements, below MAX_STRIDE), and whether two stretches of memory meet.
inline size_t rows_bytes(size_t n1, size_t s1, size_t n2, size_t s2, size_t element) {
    return n1 && n2 ? ((n1 - 1) * s1 + (n2 - 1) * s2 + HD) * element : 0;
}
inline bool stretches_meet(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a_bytes && b_bytes && (x < y ? y - x < a_bytes : x - y < b_bytes);
}

// kq8_write_kv / kq8_read_kv: rows of K and V outside the cache (element
// strides, elements of a row adjacent) and the slot of each token.
struct RowsParams {
    kq8_cache_t cache;
    void* k;
    void* v;
    int64_t k_st, k_sh, v_st, v_sh;
    const int32_t* slot;
    int32_t T;
    uint32_t* status;
};

// kq8_tree_commit
struct CommitParams {
    kq8_cache_t cache;
    const int32_t* page_table;
    int32_t max_pages;
    const int32_t* base_lens;
    const int32_t* path;
    const int32_t* path_len;
    int32_t max_path;
    uint32_t* status;
};

// Shared argument checks of a kq8_cache_t (head_dim 128, kv_bs a multiple of
// 32 up to 256, 16-byte aligned arrays); returns a KQ8_ERR_* code or KQ8_OK.
int check_cache_args(const kq8_cache_t* c);

// The V array as the 3-D tensor map the attention kernels copy sub-tiles
// through (see AttnParams::vmap); returns a KQ8_ERR_* code or KQ8_OK.
int encode_vmap(CUtensorMap* map, const kq8_cache_t& c, bool q4);
// cuTensorMapEncodeTiled for the library's other maps: rank, sizes, strides
// (bytes, from dimension 1) and box of a tensor of `type`, with `swizzle`.
int encode_tensor_map(CUtensorMap* map, CUtensorMapDataType type, uint32_t rank, void* base,
                      const uint64_t* dims, const uint64_t* strides, const uint32_t* box,
                      CUtensorMapSwizzle swizzle);
// SMs of the current device (152 without one).
int device_sms();

// A programmatic launch of `kern` with `smem` bytes of dynamic shared memory.  The
// opt-in to more than 48 KB is made once per kernel and device (it costs as much as
// a launch).
template <typename... KArgs, typename... Args>
int launch_smem(void (*kern)(KArgs...), std::atomic<uint64_t>& opted, dim3 grid, int threads,
                size_t smem, cudaStream_t stream, Args... args) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return KQ8_ERR_CUDA;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!(opted.load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
            cudaSuccess)
            return KQ8_ERR_CUDA;
        opted.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) return KQ8_ERR_CUDA;
    return cudaPeekAtLastError() == cudaSuccess ? KQ8_OK : KQ8_ERR_CUDA;
}

int launch_append(const kq8_cache_t& c, const float* k, const float* v, const int32_t* slot,
                  int32_t T, uint32_t* status, cudaStream_t stream);
int launch_append_q4(const kq8_cache_t& c, const float* k, const float* v, const int32_t* slot,
                     int32_t T, uint32_t* status, cudaStream_t stream);
int launch_debug_quantize(int8_t* qi, float* qsc, const float* q, int32_t rows, cudaStream_t s);
int launch_debug_dots(int32_t* dots, const float* q, const kq8_cache_t& c,
                      const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens,
                      int32_t max_seq_len, int32_t B, int32_t nq, cudaStream_t s);

// Attention over KV chunks (+ the merge when any sequence spans > 1 chunk).
int launch_attn(const AttnParams& p, int G, bool sparse, int B, int nkv, cudaStream_t s);
int launch_attn_q4(const AttnParams& p, int G, int B, int nkv, cudaStream_t s);
int launch_attn_withhold(const AttnParams& p, int G, int B, int nkv, cudaStream_t s);
int launch_probe(const SparseParams& p, int G, int B, int nkv, cudaStream_t s);
int launch_state_reset(float* acc, float2* ms, int rows, cudaStream_t s);
int launch_state_finalize(float* out, const float* acc, const float2* ms, int rows, cudaStream_t s);
int launch_state_merge(float* acc, float2* ms, const float* pacc, const float2* pms, int parts,
                       int rows, cudaStream_t s);
int probe_blocks_per_cta(int block, int kv_bs);
int launch_prefill(const PrefillParams& p, int G, int nkv, cudaStream_t s);
int launch_prefill_rows(int32_t* row_seq, int32_t* row_len, const int32_t* q_off,
                        const int32_t* seq_lens, int32_t B, int32_t total_q, int32_t max_seq_len,
                        int32_t max_q_len, cudaStream_t s);
int launch_topk(const SparseParams& p, int G, int B, int nkv, cudaStream_t s);

}  // namespace kq8
