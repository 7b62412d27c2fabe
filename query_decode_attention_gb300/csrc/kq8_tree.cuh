// kq8_tree.cuh -- what the two draft-tree attention kernels share: the call's
// parameters, the query and output types, the tree mask.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "kq8_common.cuh"

namespace kq8 {

constexpr float TR_LOG2E = 1.4426950408889634f;
constexpr size_t TR_STATUS_BYTES = 256;
constexpr size_t TR_COUNTERS = 16384;
constexpr size_t TR_HEADER = TR_STATUS_BYTES + TR_COUNTERS * sizeof(uint32_t);

struct TreeParams {
    CUtensorMap vmap;
    void* out;
    const void* q;
    int64_t q_st, q_sh;  // element strides of q's tokens and heads
    int32_t dtype;
    int32_t total_q;
    kq8_cache_t cache;
    const int32_t* page_table;
    int32_t max_pages;
    const int32_t* seq_lens;
    const int32_t* q_off;
    const uint32_t* mask;  // [total_q][mask_words]; null: node i sees nodes 0 .. i
    int32_t mask_words;
    int32_t max_seq_len, max_q_len;
    int32_t b0, seqs;      // sequences of this launch
    int32_t nq, G;
    float scale;
    int32_t chunk_tiles, num_chunks, row_tiles;
    float* part_acc;
    float* spill;          // tensor cores, hi and lo parts: [CTA][2][HD][128]
    float2* part_ms;       // the same places, without HD
    uint32_t* status;      // [0] status bits, [1] set by a CTA that gave up
    uint32_t* counters;    // [pairs]
};

__device__ __forceinline__ float tr_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 4 elements of a q row as fp32 (exact).
__device__ __forceinline__ float4 load_q4(const void* q, int dtype, int64_t at) {
    if (dtype == KQ8_F32) return *reinterpret_cast<const float4*>(static_cast<const float*>(q) + at);
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(q) + at);
    if (dtype == KQ8_F16) {
        const float2 a = h2_to_f2(w.x), b = h2_to_f2(w.y);
        return make_float4(a.x, a.y, b.x, b.y);
    }
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
}
// load(type code as a constant) for the call's type: bf16, or with hi and lo parts fp32
// or fp16.  A batch of loads behind one branch stays in flight together.
template <bool HILO, typename F>
__device__ __forceinline__ void load_type(int dtype, F&& load) {
    if (!HILO)
        load(std::integral_constant<int, KQ8_BF16>{});
    else if (dtype == KQ8_F32)
        load(std::integral_constant<int, KQ8_F32>{});
    else
        load(std::integral_constant<int, KQ8_F16>{});
}
// One rounding to the output type.
__device__ __forceinline__ void store_out4(void* out, int dtype, size_t at, const float4 x) {
    if (dtype == KQ8_F32) {
        *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = x;
    } else if (dtype == KQ8_F16) {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) =
            make_uint2(f2_to_h2(x.x, x.y), f2_to_h2(x.z, x.w));
    } else {
        __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) =
            make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
    }
}

// What node i of a sequence with nb nodes sees among nodes jt .. jt + 31, as
// bits; a negative node index is a committed token (always seen), one past the
// last node never is.
__device__ __forceinline__ uint32_t node_window(const TreeParams& P, int64_t row0, int i, int nb,
                                                int jt) {
    auto word = [&](int w) -> uint32_t {
        if (w < 0) return 0xFFFFFFFFu;
        const int j0 = 32 * w;
        if (j0 >= nb) return 0u;
        uint32_t x;
        if (P.mask)
            x = P.mask[(row0 + i) * P.mask_words + w];
        else
            x = i >= j0 + 31 ? 0xFFFFFFFFu : (i < j0 ? 0u : (2u << (i - j0)) - 1u);
        return nb >= j0 + 32 ? x : x & ((1u << (nb - j0)) - 1u);
    };
    const int w = jt >> 5, s = jt & 31;  // floor division
    return __funnelshift_r(word(w), s ? word(w + 1) : 0u, s);
}

// kq8_tree_tc.cu: the call on the tcgen05 tensor cores.  tile_rows is 128 or 256 (bf16
// only); part_acc / part_ms hold 2 * ctas * tile_rows rows.
int launch_tree_tc(const TreeParams& p, int tile_rows, int ctas, cudaStream_t s);

}  // namespace kq8
