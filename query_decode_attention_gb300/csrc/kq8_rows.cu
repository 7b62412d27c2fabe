// kq8_rows.cu -- cache rows in and out: the write path for fp32 / fp16 / bf16
// rows of any stride (article 9-3 §2, kv_quantize_per_head), the read back, and
// the move of a draft tree's accepted path to its place behind the committed
// tokens.
//
// Write and read.  A row is one (token, KV head) pair's 128 elements of K or V.
// A block takes 32 consecutive tokens of one KV head: with consecutive slots
// that is one K sub-tile and 32 V rows, 4 KB each, so every line of the pool
// that the block touches it touches whole.  Within the block, group i of lanes
// takes token krow(i): the groups of a warp then hold K rows at adjacent
// positions of the sub-tile (32 bytes per position and element block).  A lane
// holds 8 consecutive elements per chunk: one 16-byte access of a 16-bit row (one
// of 32 bytes of an fp32 row) and one 8-byte (q4: 4-byte) access of the pool, so
// a packed q4 word (elements e .. e + 3 low, e + 4 .. e + 7 high) never crosses
// lanes.  Both are bound by HBM: nothing is read or written twice.
//
// Measured, 8 KV heads, against a copy's 6.8 TB/s: fp32, 32768 tokens: write 52 us
// = 6.4 TB/s, read 55 us = 6.1 (68 with two 16-byte stores a lane, which fill half
// a sector row each).  bf16, 131072 tokens: read 127 us = 6.4 TB/s, write 166 us =
// 4.9: the absolute maximum, the division's reciprocal and the rounding of a row
// cost what an fp32 row's do while the bytes are half.  q4, 131072: read 104 us =
// 6.5, write 182 us = 3.7.  One token, or 64: 7.5 us, a launch's latency.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kq8_internal.h"
#include "kq8_quant.cuh"

namespace kq8 {

namespace {

constexpr int RW_LPR = 8;                 // lanes per row
constexpr int RW_NC = HD / 8 / RW_LPR;    // 8-element chunks per lane
constexpr int RW_THREADS = TILE * RW_LPR; // 32 tokens of one KV head

struct Elem8 {
    float4 a, b;
};

// 8 consecutive elements as they lie in memory, one 16-byte word (fp32: two).
// VEC: p is aligned to their 16 (32) bytes; else element by element.
template <typename E>
struct Raw8 {
    static constexpr int W = (int)sizeof(E) * 8 / 16;
    uint4 w[W];
};
template <typename E, bool VEC>
__device__ __forceinline__ Raw8<E> load8(const E* p) {
    union {
        Raw8<E> r;
        E e[8];
    } u;
    if constexpr (VEC) {
        if constexpr (sizeof(E) == 4)
            asm volatile("ld.global.cs.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(u.r.w[0].x), "=r"(u.r.w[0].y), "=r"(u.r.w[0].z), "=r"(u.r.w[0].w),
                           "=r"(u.r.w[1].x), "=r"(u.r.w[1].y), "=r"(u.r.w[1].z), "=r"(u.r.w[1].w)
                         : "l"(p));
        else
            u.r.w[0] = __ldcs(reinterpret_cast<const uint4*>(p));
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) u.e[i] = p[i];
    }
    return u.r;
}
__device__ __forceinline__ float2 pair_f32(uint32_t w, __half) { return h2_to_f2(w); }
__device__ __forceinline__ float2 pair_f32(uint32_t w, __nv_bfloat16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// As fp32 (exact).
template <typename E>
__device__ __forceinline__ Elem8 widen(const Raw8<E>& r) {
    Elem8 x;
    if constexpr (sizeof(E) == 4) {
        x.a = *reinterpret_cast<const float4*>(&r.w[0]);
        x.b = *reinterpret_cast<const float4*>(&r.w[1]);
    } else {
        const float2 p = pair_f32(r.w[0].x, E()), q = pair_f32(r.w[0].y, E());
        const float2 s = pair_f32(r.w[0].z, E()), t = pair_f32(r.w[0].w, E());
        x.a = make_float4(p.x, p.y, q.x, q.y);
        x.b = make_float4(s.x, s.y, t.x, t.y);
    }
    return x;
}
// max |x| of the 8, NaN ignored as by fmaxf; 16-bit elements in pairs.
__device__ __forceinline__ uint32_t pair_max(uint32_t a, uint32_t b, __half) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7FFF7FFFu), "r"(b & 0x7FFF7FFFu));
    return r;
}
__device__ __forceinline__ uint32_t pair_max(uint32_t a, uint32_t b, __nv_bfloat16) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7FFF7FFFu), "r"(b & 0x7FFF7FFFu));
    return r;
}
template <typename E>
__device__ __forceinline__ float max8(const Raw8<E>& r) {
    if constexpr (sizeof(E) == 4) {
        const Elem8 x = widen<E>(r);
        return fmaxf(absmax4(x.a), absmax4(x.b));
    } else {
        const uint32_t m = pair_max(pair_max(r.w[0].x, r.w[0].y, E()),
                                    pair_max(r.w[0].z, r.w[0].w, E()), E());
        const float2 f = pair_f32(m, E());
        return fmaxf(fmaxf(f.x, f.y), 0.0f);  // (four NaN pairs)
    }
}
// Stored with one rounding each.
__device__ __forceinline__ uint32_t pair_of(float x, float y, __half) { return f2_to_h2(x, y); }
__device__ __forceinline__ uint32_t pair_of(float x, float y, __nv_bfloat16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename E, bool VEC>
__device__ __forceinline__ void store8(E* p, const float (&x)[8]) {
    union {
        Raw8<E> r;
        E e[8];
    } u;
    if constexpr (sizeof(E) == 4) {
#pragma unroll
        for (int i = 0; i < 8; i++) u.e[i] = x[i];
    } else {
        u.r.w[0] = make_uint4(pair_of(x[0], x[1], E()), pair_of(x[2], x[3], E()),
                              pair_of(x[4], x[5], E()), pair_of(x[6], x[7], E()));
    }
    if constexpr (VEC && sizeof(E) == 4) {
        // whole 32-byte sectors: two 16-byte stores a lane apart in a row half fill them
        asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p),
                     "r"(u.r.w[0].x), "r"(u.r.w[0].y), "r"(u.r.w[0].z), "r"(u.r.w[0].w),
                     "r"(u.r.w[1].x), "r"(u.r.w[1].y), "r"(u.r.w[1].z), "r"(u.r.w[1].w)
                     : "memory");
    } else if constexpr (VEC) {
        __stcs(reinterpret_cast<uint4*>(p), u.r.w[0]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) p[i] = u.e[i];
    }
}

// Where row r (0 .. kv_bs - 1) of (page, head) keeps elements e .. e + 7 (e a
// multiple of 8): byte offsets into the K and V arrays.
template <int BITS>
__device__ __forceinline__ size_t k_off(int32_t page, int h, int nkv, int kv_bs, int r, int e) {
    if constexpr (BITS == 8)
        return kv_sub_off(page, h, nkv, kv_bs, r / TILE) + (size_t)(e >> 5) * 1024 +
               (size_t)kpos(r % TILE) * 32 + (e & 31);
    else
        return kv4_sub_off(page, h, nkv, kv_bs, r / TILE) + (size_t)(e >> 5) * 512 +
               (size_t)kpos(r % TILE) * 16 + ((e & 31) >> 1);
}
template <int BITS>
__device__ __forceinline__ size_t v_off(int32_t page, int h, int nkv, int kv_bs, int r, int e) {
    constexpr int ROW = BITS == 8 ? HD : HD / 2;
    return (page_head(page, h, nkv) * (size_t)kv_bs + (size_t)r) * ROW + (BITS == 8 ? e : e / 2);
}

// Where a slot is: page and row; false (and a status bit for a slot past the pool)
// where there is nothing to do.  Every lane of a group gets the same answer.
__device__ __forceinline__ bool slot_at(const RowsParams& P, int32_t sl, int32_t& page, int& r) {
    if (sl < 0) return false;
    if ((int64_t)sl >= (int64_t)P.cache.num_pages * P.cache.kv_bs) {
        if (threadIdx.x % RW_LPR == 0 && P.status) atomicOr(P.status, KQ8_STATUS_BAD_SLOT);
        return false;
    }
    page = sl / P.cache.kv_bs;
    r = sl - page * P.cache.kv_bs;
    return true;
}

template <int BITS>
__device__ __forceinline__ void put_codes(int8_t* dst, const Elem8& x, float d, float r, bool zero) {
    constexpr float TOP = BITS == 8 ? 127.0f : 7.0f;
    constexpr int OFF = BITS == 8 ? 0 : 8;
    uint32_t lo = BITS == 8 ? 0u : 0x08080808u, hi = lo;
    if (!zero) {
        lo = quantize4(x.a, d, r, -TOP, TOP, OFF);
        hi = quantize4(x.b, d, r, -TOP, TOP, OFF);
    }
    if constexpr (BITS == 8)
        *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
    else
        *reinterpret_cast<uint32_t*>(dst) = lo | (hi << 4);
}

// The write rule on the row widened to fp32, so the codes and maxima equal
// kq8_append_kv's for the same values bit for bit.  The rows are fetched beside
// their slots; a block takes NT sub-tiles of 32 tokens, all fetched before the first
// is quantised.
template <typename E, int BITS, bool VEC, int NT>
__global__ void __launch_bounds__(RW_THREADS) kq8_write_kernel(const RowsParams P) {
    griddep_wait();
    griddep_launch_dependents();
    const int j = threadIdx.x % RW_LPR, h = blockIdx.y;
    const int64_t t0 = (int64_t)blockIdx.x * (NT * TILE) + krow(threadIdx.x / RW_LPR);
    const int nkv = P.cache.num_kv_heads, kv_bs = P.cache.kv_bs;
    int32_t slot[NT];
    Raw8<E> x[NT][2][RW_NC];
#pragma unroll
    for (int n = 0; n < NT; n++) {
        const int64_t t = t0 + n * TILE;
        slot[n] = t < P.T ? __ldg(P.slot + t) : -1;
        if (t < P.T) {
            const E* k = static_cast<const E*>(P.k) + t * P.k_st + h * P.k_sh;
            const E* v = static_cast<const E*>(P.v) + t * P.v_st + h * P.v_sh;
#pragma unroll
            for (int i = 0; i < RW_NC; i++) {
                x[n][0][i] = load8<E, VEC>(k + 8 * (RW_LPR * i + j));
                x[n][1][i] = load8<E, VEC>(v + 8 * (RW_LPR * i + j));
            }
        } else {
#pragma unroll
            for (int s = 0; s < 2; s++)
#pragma unroll
                for (int i = 0; i < RW_NC; i++)
#pragma unroll
                    for (int w = 0; w < Raw8<E>::W; w++) x[n][s][i].w[w] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
#pragma unroll
    for (int n = 0; n < NT; n++) {
        float m[2];
#pragma unroll
        for (int s = 0; s < 2; s++) {
            m[s] = 0.0f;
#pragma unroll
            for (int i = 0; i < RW_NC; i++) m[s] = fmaxf(m[s], max8<E>(x[n][s][i]));
#pragma unroll
            for (int o = 1; o < RW_LPR; o <<= 1)
                m[s] = fmaxf(m[s], __shfl_xor_sync(0xffffffffu, m[s], o));
        }
        int32_t page;
        int r;
        if (!slot_at(P, slot[n], page, r)) continue;
#pragma unroll
        for (int s = 0; s < 2; s++) {
            const float d = __fmul_rn(m[s], BITS == 8 ? inv127() : inv7()), rcp = __frcp_rn(d);
#pragma unroll
            for (int i = 0; i < RW_NC; i++) {
                const int e = 8 * (RW_LPR * i + j);
                int8_t* dst = s == 0 ? P.cache.k + k_off<BITS>(page, h, nkv, kv_bs, r, e)
                                     : P.cache.v + v_off<BITS>(page, h, nkv, kv_bs, r, e);
                put_codes<BITS>(dst, widen<E>(x[n][s][i]), d, rcp, m[s] == 0.0f);
            }
        }
        if (j == 0) {
            const size_t so = page_head(page, h, nkv) * (size_t)kv_bs + r;
            P.cache.kscale[so] = m[0];
            P.cache.vscale[so] = m[1];
        }
    }
}

// 8 codes as stored, and as fp32 (exact).
template <int BITS>
struct Codes8 {
    uint32_t w[BITS == 8 ? 2 : 1];
};
template <int BITS>
__device__ __forceinline__ Codes8<BITS> get_codes(const int8_t* src) {
    Codes8<BITS> c;
    if constexpr (BITS == 8) {
        const uint2 w = __ldcs(reinterpret_cast<const uint2*>(src));
        c.w[0] = w.x;
        c.w[1] = w.y;
    } else {
        c.w[0] = __ldcs(reinterpret_cast<const uint32_t*>(src));
    }
    return c;
}
template <int BITS>
__device__ __forceinline__ void code_values(const Codes8<BITS>& c, float (&y)[8]) {
    if constexpr (BITS == 8) {
        i8x4_to_f32(c.w[0], y[0], y[1], y[2], y[3]);
        i8x4_to_f32(c.w[1], y[4], y[5], y[6], y[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            y[i] = (float)((int)((c.w[0] >> (8 * (i & 3) + 4 * (i >> 2))) & 15u) - 8);
    }
}

// The values the rows stand for: code * (stored max * (1/127)) (q4: 1/7), one
// fp32 product as the attention kernels' readers form it, then one rounding to
// the output type.  NT as for the write.
template <typename E, int BITS, bool VEC, int NT>
__global__ void __launch_bounds__(RW_THREADS) kq8_read_kernel(const RowsParams P) {
    griddep_wait();
    griddep_launch_dependents();
    const int j = threadIdx.x % RW_LPR, h = blockIdx.y;
    const int64_t t0 = (int64_t)blockIdx.x * (NT * TILE) + krow(threadIdx.x / RW_LPR);
    const int nkv = P.cache.num_kv_heads, kv_bs = P.cache.kv_bs;
    int32_t slot[NT];
#pragma unroll
    for (int n = 0; n < NT; n++) slot[n] = t0 + n * TILE < P.T ? __ldg(P.slot + t0 + n * TILE) : -1;
    bool on[NT];
    Codes8<BITS> c[NT][2][RW_NC];
    float m[NT][2];
#pragma unroll
    for (int n = 0; n < NT; n++) {
        int32_t page;
        int r;
        on[n] = slot_at(P, slot[n], page, r);
        if (!on[n]) continue;
#pragma unroll
        for (int i = 0; i < RW_NC; i++) {
            const int e = 8 * (RW_LPR * i + j);
            c[n][0][i] = get_codes<BITS>(P.cache.k + k_off<BITS>(page, h, nkv, kv_bs, r, e));
            c[n][1][i] = get_codes<BITS>(P.cache.v + v_off<BITS>(page, h, nkv, kv_bs, r, e));
        }
        const size_t so = page_head(page, h, nkv) * (size_t)kv_bs + r;
        m[n][0] = P.cache.kscale[so];
        m[n][1] = P.cache.vscale[so];
    }
#pragma unroll
    for (int n = 0; n < NT; n++) {
        if (!on[n]) continue;
        const int64_t t = t0 + n * TILE;
        E* dst[2] = {static_cast<E*>(P.k) + t * P.k_st + h * P.k_sh,
                     static_cast<E*>(P.v) + t * P.v_st + h * P.v_sh};
#pragma unroll
        for (int s = 0; s < 2; s++) {
            const float d = __fmul_rn(m[n][s], BITS == 8 ? inv127() : inv7());
#pragma unroll
            for (int i = 0; i < RW_NC; i++) {
                float y[8];
                code_values<BITS>(c[n][s][i], y);
#pragma unroll
                for (int k = 0; k < 8; k++) y[k] = __fmul_rn(y[k], d);
                store8<E, VEC>(dst[s] + 8 * (RW_LPR * i + j), y);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The accepted path of a draft tree: of sequence b's drafts, which sit at
// positions base .. in the order they were written, draft path[i] moves to
// position base + i, for i < len.  The path ascends strictly (a tree's nodes
// follow their parents), so path[i] >= i: a block that takes the rows in order,
// a batch at a time, loads a batch before it stores it, and never stores over a
// row that a later batch loads (its sources lie at or behind the batch's own
// first position, and every earlier store before it).  Codes and maxima move
// bit for bit.  One block per (sequence, KV head); 16 lanes move a row: lanes
// 0-7 K, 8-15 V, a 16-byte (q4: 8-byte) piece each.
// A path with a bad entry, position or page moves nothing and sets a status
// bit; every block of the sequence checks the whole path, so all agree.
// A launch's latency bounds it (a path has a few rows, 264 bytes each and head).
// ---------------------------------------------------------------------------
constexpr int CM_THREADS = 256;
constexpr int CM_ROWS = CM_THREADS / 16;

template <int BITS>
__global__ void __launch_bounds__(CM_THREADS) kq8_commit_kernel(const CommitParams P) {
    griddep_wait();
    griddep_launch_dependents();
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    const int nkv = P.cache.num_kv_heads, kv_bs = P.cache.kv_bs;
    const int32_t base = P.base_lens[b], len = P.path_len[b];
    const int64_t room = (int64_t)P.max_pages * kv_bs;
    const int32_t* path = P.path + (size_t)b * P.max_path;
    const int32_t* table = P.page_table + (size_t)b * P.max_pages;
    uint32_t bad = 0;
    if (base < 0 || len < 0 || len > P.max_path) {
        bad = KQ8_STATUS_BAD_SEQLEN;
    } else {
        for (int i = tid; i < len; i += CM_THREADS) {
            const int32_t j = path[i];
            if (j < 0 || (i > 0 && path[i - 1] >= j) || (int64_t)base + j >= room) {
                bad |= KQ8_STATUS_BAD_SEQLEN;
                continue;
            }
            const int32_t p0 = table[(base + j) / kv_bs];
            if (p0 < 0 || p0 >= P.cache.num_pages) bad |= KQ8_STATUS_BAD_PAGE;
            if ((int64_t)base + i < room) {  // j >= i on a good path
                const int32_t p1 = table[(base + i) / kv_bs];
                if (p1 < 0 || p1 >= P.cache.num_pages) bad |= KQ8_STATUS_BAD_PAGE;
            }
        }
    }
    if (bad && P.status) atomicOr(P.status, bad);
    if (__syncthreads_or(bad != 0)) return;
    using Piece = typename std::conditional<BITS == 8, uint4, uint2>::type;
    const int l = tid & 15, e = (l & 7) * 16;  // this lane's 16 elements
    for (int i0 = 0; i0 < len; i0 += CM_ROWS) {
        const int i = i0 + (tid >> 4);
        const int32_t j = i < len ? path[i] : i;
        const bool moves = j != i;
        Piece piece;
        float scale = 0.0f;
        auto place = [&](int32_t pos, int8_t*& codes, float*& s) {
            const int32_t page = table[pos / kv_bs];
            const int r = pos % kv_bs;
            codes = l < 8 ? P.cache.k + k_off<BITS>(page, h, nkv, kv_bs, r, e)
                          : P.cache.v + v_off<BITS>(page, h, nkv, kv_bs, r, e);
            s = (l < 8 ? P.cache.kscale : P.cache.vscale) +
                page_head(page, h, nkv) * (size_t)kv_bs + r;
        };
        int8_t* codes;
        float* s;
        if (moves) {
            place(base + j, codes, s);
            piece = *reinterpret_cast<const Piece*>(codes);
            if ((l & 7) == 0) scale = *s;
        }
        __syncthreads();  // the batch is loaded before any of it is stored
        if (moves) {
            place(base + i, codes, s);
            *reinterpret_cast<Piece*>(codes) = piece;
            if ((l & 7) == 0) *s = scale;
        }
        __syncthreads();  // stored before the next batch loads
    }
}

template <bool WRITE, typename E, int BITS, bool VEC, int NT>
int launch_rows_n(const RowsParams& p, cudaStream_t s) {
    const dim3 grid((unsigned)(((int64_t)p.T + NT * TILE - 1) / (NT * TILE)),
                    (unsigned)p.cache.num_kv_heads);
    if constexpr (WRITE)
        return launch_pdl(kq8_write_kernel<E, BITS, VEC, NT>, grid, RW_THREADS, s, p);
    else
        return launch_pdl(kq8_read_kernel<E, BITS, VEC, NT>, grid, RW_THREADS, s, p);
}
template <bool WRITE, typename E, int BITS>
int launch_rows_t(const RowsParams& p, bool vec, cudaStream_t s) {
    if (!vec) return launch_rows_n<WRITE, E, BITS, false, 1>(p, s);
    // A bulk read of 16-bit rows takes two sub-tiles a block, their loads in flight
    // together (131072 tokens, 8 KV heads, bf16: 141 us with one, 127 with two, 149 with
    // four).  A small one has too few blocks for that; a write holds more registers per
    // sub-tile (183, 212, 303 us), fp32 rows and q4 codes gain nothing.
    if constexpr (!WRITE && BITS == 8 && sizeof(E) == 2) {
        const int64_t blocks = ((int64_t)p.T + TILE - 1) / TILE * p.cache.num_kv_heads;
        if (blocks >= (int64_t)device_sms() * 16) return launch_rows_n<WRITE, E, BITS, true, 2>(p, s);
    }
    return launch_rows_n<WRITE, E, BITS, true, 1>(p, s);
}

template <bool WRITE, int BITS>
int launch_rows(const RowsParams& p, int dtype, bool vec, cudaStream_t s) {
    switch (dtype) {
        case KQ8_F32: return launch_rows_t<WRITE, float, BITS>(p, vec, s);
        case KQ8_F16: return launch_rows_t<WRITE, __half, BITS>(p, vec, s);
        default: return launch_rows_t<WRITE, __nv_bfloat16, BITS>(p, vec, s);
    }
}

// Whether n1 x n2 rows of HD elements at strides s1 and s2 do not overlap (the
// larger stride steps over all rows of the smaller one).
bool rows_apart(int64_t s1, int64_t n1, int64_t s2, int64_t n2) {
    if (n1 <= 1) return n2 <= 1 || s2 >= HD;
    if (n2 <= 1) return s1 >= HD;
    if (s1 > s2) return rows_apart(s2, n2, s1, n1);
    return s1 >= HD && s2 >= (n1 - 1) * s1 + HD;
}

// Whether two sets of such rows (each apart in itself) that lie `d` >= 0 elements from
// each other are apart too: a row of one meets a row of the other only if d is within
// HD of a difference i * s1 + j * s2, |i| < n1, |j| < n2, and of those only the nearest
// ones can be.
bool rows_interleave(int64_t d, int64_t s1, int64_t n1, int64_t s2, int64_t n2) {
    if (n1 <= 1) s1 = 0;
    if (n2 <= 1) s2 = 0;
    if (s1 < s2) return rows_interleave(d, s2, n2, s1, n1);
    const int64_t i0 = s1 ? d / s1 : 0;
    for (int64_t i = i0; i <= i0 + 1 && i < n1; i++) {
        const int64_t r = d > i * s1 ? d - i * s1 : i * s1 - d, j0 = s2 ? r / s2 : 0;
        for (int64_t j = j0; j <= j0 + 1 && j < n2; j++)
            if ((r > j * s2 ? r - j * s2 : j * s2 - r) < HD) return false;
    }
    return true;
}

// Checks, the choice of vector accesses (bases and strides multiples of 8
// elements), launch.
template <bool WRITE>
int rows_impl(const kq8_cache_t* cache, int32_t bits, void* k, void* v, int32_t dtype,
              size_t k_st, size_t k_sh, size_t v_st, size_t v_sh, const int32_t* slot, int32_t T,
              uint32_t* status, kq8_stream_t stream) {
    int rc = check_cache_args(cache);
    if (rc) return rc;
    if (bits != 8 && bits != 4) return KQ8_ERR_UNSUPPORTED;
    if (dtype != KQ8_F32 && dtype != KQ8_F16 && dtype != KQ8_BF16) return KQ8_ERR_UNSUPPORTED;
    if (cache->num_kv_heads > 65535) return KQ8_ERR_UNSUPPORTED;
    if (T < 0) return KQ8_ERR_INVALID_ARG;
    if (T == 0) return KQ8_OK;
    const size_t es = dtype == KQ8_F32 ? 4 : 2;
    if (!k || !v || !slot || (uintptr_t)k % es || (uintptr_t)v % es || (uintptr_t)slot % 4)
        return KQ8_ERR_INVALID_ARG;
    if (status && (uintptr_t)status % 4) return KQ8_ERR_INVALID_ARG;
    const size_t st[4] = {k_st, k_sh, v_st, v_sh};
    const size_t chunk = 8 * es;  // what a lane moves at a time
    bool vec = (uintptr_t)k % chunk == 0 && (uintptr_t)v % chunk == 0;
    for (size_t x : st) {
        if (x > MAX_STRIDE) return KQ8_ERR_INVALID_ARG;
        vec = vec && (x * es) % chunk == 0;
    }
    // the rows a read stores must not overlap
    const int64_t heads = cache->num_kv_heads;
    if (!WRITE) {
        if (!rows_apart((int64_t)k_st, T, (int64_t)k_sh, heads) ||
            !rows_apart((int64_t)v_st, T, (int64_t)v_sh, heads))
            return KQ8_ERR_INVALID_ARG;
        if (stretches_meet(k, rows_bytes(T, k_st, heads, k_sh, es), v,
                           rows_bytes(T, v_st, heads, v_sh, es))) {
            const bool same = (T == 1 || k_st == v_st) && (heads == 1 || k_sh == v_sh);
            const uintptr_t x = (uintptr_t)k, y = (uintptr_t)v;
            if (!same || !rows_interleave((int64_t)((x < y ? y - x : x - y) / es), (int64_t)k_st, T,
                                          (int64_t)k_sh, heads))
                return KQ8_ERR_INVALID_ARG;
        }
    }
    RowsParams p;
    p.cache = *cache;
    p.k = k;
    p.v = v;
    p.k_st = (int64_t)k_st;
    p.k_sh = (int64_t)k_sh;
    p.v_st = (int64_t)v_st;
    p.v_sh = (int64_t)v_sh;
    p.slot = slot;
    p.T = T;
    p.status = status;
    return bits == 8 ? launch_rows<WRITE, 8>(p, dtype, vec, (cudaStream_t)stream)
                     : launch_rows<WRITE, 4>(p, dtype, vec, (cudaStream_t)stream);
}

}  // namespace
}  // namespace kq8

using namespace kq8;

extern "C" {

int kq8_write_kv(const kq8_cache_t* cache, int32_t bits, const void* k, const void* v,
                 int32_t dtype, size_t k_token_stride, size_t k_head_stride,
                 size_t v_token_stride, size_t v_head_stride, const int32_t* slot, int32_t T,
                 uint32_t* status, kq8_stream_t stream) {
    return rows_impl<true>(cache, bits, const_cast<void*>(k), const_cast<void*>(v), dtype,
                           k_token_stride, k_head_stride, v_token_stride, v_head_stride, slot, T,
                           status, stream);
}

int kq8_read_kv(const kq8_cache_t* cache, int32_t bits, void* k, void* v, int32_t dtype,
                size_t k_token_stride, size_t k_head_stride, size_t v_token_stride,
                size_t v_head_stride, const int32_t* slot, int32_t T, uint32_t* status,
                kq8_stream_t stream) {
    return rows_impl<false>(cache, bits, k, v, dtype, k_token_stride, k_head_stride,
                            v_token_stride, v_head_stride, slot, T, status, stream);
}

int kq8_tree_commit(const kq8_cache_t* cache, int32_t bits, const int32_t* page_table,
                    int32_t max_pages, const int32_t* base_lens, const int32_t* path,
                    const int32_t* path_len, int32_t max_path, int32_t B, uint32_t* status,
                    kq8_stream_t stream) {
    int rc = check_cache_args(cache);
    if (rc) return rc;
    if (bits != 8 && bits != 4) return KQ8_ERR_UNSUPPORTED;
    if (B < 0 || max_path < 0 || max_pages < 0) return KQ8_ERR_INVALID_ARG;
    if (B > 65535 || (int64_t)max_pages * cache->kv_bs >= (1 << 29)) return KQ8_ERR_UNSUPPORTED;
    if (status && (uintptr_t)status % 4) return KQ8_ERR_INVALID_ARG;
    if (B == 0 || max_path == 0) return KQ8_OK;
    if (!page_table || !base_lens || !path || !path_len) return KQ8_ERR_INVALID_ARG;
    CommitParams p;
    p.cache = *cache;
    p.page_table = page_table;
    p.max_pages = max_pages;
    p.base_lens = base_lens;
    p.path = path;
    p.path_len = path_len;
    p.max_path = max_path;
    p.status = status;
    const dim3 grid((unsigned)cache->num_kv_heads, (unsigned)B);
    return bits == 8 ? launch_pdl(kq8_commit_kernel<8>, grid, CM_THREADS, (cudaStream_t)stream, p)
                     : launch_pdl(kq8_commit_kernel<4>, grid, CM_THREADS, (cudaStream_t)stream, p);
}

}  // extern "C"
