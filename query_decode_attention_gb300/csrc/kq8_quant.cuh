// kq8_quant.cuh -- the write rule's rounding (article 9-3 §2) and the programmatic
// launch, shared by the kernels that write and move cache rows.
#pragma once

#include "kq8_common.cuh"

namespace kq8 {

// max that is NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// roundf(x / d) for the elements of a row whose step is d, |x / d| < 128, with
// r = RN(1 / d).  r and the product q = RN(x * r) each round once (relative
// 2^-24), so |q - x / d| <= 128 * 2^-23 and |fl(x / d) - x / d| <= 2^-18:
// q is within 2^-15.5 of the IEEE quotient fl(x / d).  Unless q lies within
// 2^-14 of a half-integer both therefore round to the same integer, and the
// nearest integer to q (no tie possible) is roundf(fl(x / d)).  The rare
// near-half case (about 1 in 8000 elements), and a non-finite q (d subnormal
// or 0), take the IEEE quotient itself, so the result always equals the
// method's roundf(x / d) bit for bit.
// The nearest integer comes from adding 1.5 * 2^23 + off (exact for |q| < 2^22):
// the sum's low byte is then (n + off) mod 256, the code byte itself.  On the
// fast path |q| < 127.5 (and < 7.5 for q4), so no clamp is needed there.
// Returns the lane's four code bytes (element i in byte i); r = RN(1 / d) (the
// caller computes it once per row), lo / hi clamp the slow path, off is 0 (q8,
// two's complement) or 8 (q4, offset binary).
__device__ __forceinline__ uint32_t quantize4(const float4 x, float d, float r, float lo, float hi,
                                              int off) {
    const float magic = 12582912.0f + (float)off;  // 1.5 * 2^23 + off
    const float2 r2 = make_float2(r, r), mg = make_float2(magic, magic);
    const float2 qa = __fmul2_rn(make_float2(x.x, x.y), r2), qb = __fmul2_rn(make_float2(x.z, x.w), r2);
    const float2 ta = __fadd2_rn(qa, mg), tb = __fadd2_rn(qb, mg);
    // q - (t - magic), both differences exact where they matter
    const float2 neg = make_float2(-magic, -magic), minus = make_float2(-1.0f, -1.0f);
    const float2 da = __ffma2_rn(__fadd2_rn(ta, neg), minus, qa);
    const float2 db = __ffma2_rn(__fadd2_rn(tb, neg), minus, qb);
    const float far = 0.5f - 0x1p-14f;
    const float most = max_nan(max_nan(fabsf(da.x), fabsf(da.y)), max_nan(fabsf(db.x), fabsf(db.y)));
    const bool ok = most < far;  // NaN / inf compare false
    const float t0 = ta.x, t1 = ta.y, t2 = tb.x, t3 = tb.y;
    if (ok)
        return __byte_perm(__byte_perm(__float_as_uint(t0), __float_as_uint(t1), 0x0040),
                           __byte_perm(__float_as_uint(t2), __float_as_uint(t3), 0x0040), 0x5410);
    auto slow = [&](float v) -> uint32_t {
        const float n = fminf(fmaxf(roundf(__fdiv_rn(v, d)), lo), hi);
        return (uint32_t)((int)n + off) & 0xffu;
    };
    return slow(x.x) | (slow(x.y) << 8) | (slow(x.z) << 16) | (slow(x.w) << 24);
}

__device__ __forceinline__ float absmax4(const float4 x) {
    return fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
}

// The kernels that write, read and move rows are programmatic launches: their
// CTAs may be scheduled while the kernel before them (typically the previous
// layer's attention) finishes, and wait for its completion before they read or
// write anything, so the stream order of the call's effects is unchanged; only
// the launch latency overlaps.
template <typename... KArgs, typename... Args>
inline int launch_pdl(void (*kern)(KArgs...), dim3 grid, int threads, cudaStream_t stream,
                      Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) return KQ8_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? KQ8_OK : KQ8_ERR_CUDA;
}

}  // namespace kq8
