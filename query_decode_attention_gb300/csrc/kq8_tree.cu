// kq8_tree.cu -- attention for trees of drafted tokens over the paged q8 cache.
//
// Speculative decoding writes the nb drafts of a sequence behind its committed
// tokens and asks, in one call, what every draft would attend: the committed
// tokens (base = n - nb of them) and the drafts on its own branch, given as a
// bit mask.  Each (node, query head) row is computed like one decode query
// (article 9-2 §2): Q quantised once in 32-element max-abs blocks, score =
// ((sum_b dot_b * qsc_b) * ks) * scale with exact integer block dots, a one-pass
// softmax, one divide at the end.
//
// Up to 32 rows (nodes x query heads) of a KV head; more go to kq8_tree_tc.cu.
//
// Work decomposition: CTA = (KV chunk, tile of 16 or 32 rows, KV head, sequence), 4
// warps.  The rows of a KV head are its G query heads of every node.  As in the
// decode kernel each warp owns a ring (two or three stages) of 32-token sub-tiles filled by
// bulk and tensor copies, and takes every fourth sub-tile of its chunk; chunks
// are merged by the last CTA to finish (a ticket).  Per sub-tile, on the warp's
// matrix instructions (m16n8k16, fp16 in, fp32 out):
//   scores: 4 groups of 8 tokens x 4 element blocks x 2 k-steps.  The codes of
//     Q and K are exact in fp16 and a block dot is below 2^19, so each fp32
//     accumulator is the exact integer block dot; the blocks' Q scales follow
//     as fp32 multiply-adds.
//   values: the weights p * vstep as fp16 (hi + lo, 22 significant bits, for
//     fp32 and fp16 outputs; hi alone for bf16 outputs, whose own rounding is
//     16 times coarser) times the V codes, exact in fp16.
// Token order.  Lane (g, c) of the score accumulators holds rows g, g + 8 and
// columns 2c, 2c + 1 of each 8-token group.  Column n of group i is token
//   tok(i, n) = 4 n + (i + n / 2) % 4,
// which is K position 8 ((i + n / 2) % 4) + n: the eight 32-byte pieces that a
// group reads lie in different banks, and lane c's tokens of group i are the
// two that the same lane needs for k-columns of the value product, where the
// eight V rows of a transposed 8 x 8 load are tok(i, 0..7): all different
// modulo 8, so the 128-byte swizzle keeps that load free of conflicts too.
// The weights therefore go from accumulators to operands within the lane.
// Measured, 16 x 16384 tokens, 8 KV heads (553 MB), bf16: 8 rows 101 us, 16 rows 104 us =
// 5.3 TB/s, near what HBM gives (82 us) with 12 warps an SM and the waves of chunks; 32
// rows 174 us = 3.2 TB/s, bound by latency: 8 warps an SM at 255 registers issue in a third
// of the cycles.
#include <cstring>
#include <type_traits>

#include "kq8_internal.h"
#include "kq8_tree.cuh"

namespace kq8 {
namespace {

constexpr int TR_WARPS = 4;
constexpr int TR_THREADS = TR_WARPS * 32;
constexpr int TR_MAX_CHUNK = 128;       // sub-tiles per chunk, see tree_plan
// Lazy rescale: between rescales a weight stays below 2^TR_SLACK.
constexpr float TR_SLACK = 8.0f;

// MT: tiles of 16 rows that a warp holds.  One where the rows fit it: 3 CTAs per SM
// at 168 registers; else two: every widened K and V code serves 32 rows, 2 CTAs per
// SM with a third ring stage.
template <int MT>
struct TreeShape {
    static constexpr int ROWS = 16 * MT, STAGES = MT == 1 ? 2 : 3, CTAS = MT == 1 ? 3 : 2;
};
template <int MT>
struct TreeSmem {
    static constexpr int ROWS = TreeShape<MT>::ROWS, STAGES = TreeShape<MT>::STAGES;
    // the two rings, and after the walk the warps' accumulators [warp][ROWS][HD]
    alignas(1024) uint8_t v[TR_WARPS][STAGES][SUB_V_BYTES];
    alignas(128) uint8_t k[TR_WARPS][STAGES][SUB_K_BYTES];
    alignas(16) float sc[TR_WARPS][STAGES][2][TILE];  // kscale, vscale as stored
    alignas(16) float mul[TR_WARPS][2][TILE];         // score multiplier, V step
    // Q's codes as fp16 A fragments: [16-row tile][element block][k-step][lane]
    alignas(16) uint4 qf[MT][NB][2][32];
    alignas(16) float qsc[ROWS][NB];
    alignas(16) float2 ms[TR_WARPS][ROWS];
    alignas(8) uint64_t bar[TR_WARPS][STAGES];
    int last;
};

template <int MT, bool HILO>
__global__ void __launch_bounds__(TR_THREADS, TreeShape<MT>::CTAS)
    kq8_tree_kernel(const __grid_constant__ TreeParams P) {
    constexpr int TR_ROWS = TreeShape<MT>::ROWS, TR_STAGES = TreeShape<MT>::STAGES;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    TreeSmem<MT>& S = *reinterpret_cast<TreeSmem<MT>*>(
        smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gq = lane >> 2, c4 = lane & 3;
    const int rt = blockIdx.x % P.row_tiles, chunk = blockIdx.x / P.row_tiles;
    const int h = blockIdx.y, b = P.b0 + blockIdx.z;
    const int nkv = P.cache.num_kv_heads, kv_bs = P.cache.kv_bs, subs = kv_bs / TILE;
    const int G = P.G;

    if (threadIdx.x == 0)
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.vmap))
                     : "memory");
    if (lane == 0)
        for (int s = 0; s < TR_STAGES; s++) mbar_init(&S.bar[warp][s], 1);
    fence_barrier_init();
    // nothing is read or written before the kernel before this one has
    // completed; the next one waits for this grid in the same way
    griddep_wait();
    griddep_launch_dependents();

    const int n = P.seq_lens[b];
    const int q0 = P.q_off[b];
    const int nb = P.q_off[b + 1] - q0;
    if (n < 0 || n > P.max_seq_len || nb < 0 || nb > n || nb > P.max_q_len || q0 < 0 ||
        (int64_t)q0 + nb > P.total_q) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && h == 0) atomicOr(P.status, KQ8_STATUS_BAD_SEQLEN);
        return;
    }
    const int base = n - nb;
    const int rows = min(TR_ROWS, nb * G - rt * TR_ROWS);  // of this row tile
    if (rows <= 0) return;
    const int tiles = (n + TILE - 1) / TILE;  // n >= nb >= 1 here
    const int nch = (tiles + P.chunk_tiles - 1) / P.chunk_tiles;
    if (chunk >= nch) return;
    const int ce = min(P.chunk_tiles, tiles - chunk * P.chunk_tiles);
    const int mine = ce > warp ? (ce - warp + TR_WARPS - 1) / TR_WARPS : 0;
    const int first = chunk * P.chunk_tiles + warp;  // this warp's tiles: first + 4 i

    // page ids of this warp's tiles, one per lane for a window of 32, the next
    // window fetched a window ahead
    auto load_window = [&](int w) -> int32_t {
        const int i = 32 * w + lane;
        if (i >= mine) return -1;
        const int32_t pg = P.page_table[(size_t)b * P.max_pages + (first + TR_WARPS * i) / subs];
        if (pg >= 0 && pg < P.cache.num_pages) return pg;
        atomicOr(P.status, KQ8_STATUS_BAD_PAGE);
        return -1;
    };
    int32_t page_cur = load_window(0), page_nxt = load_window(1);
    int window = 0;
    auto page_of = [&](int i) -> int32_t {
        return __shfl_sync(0xffffffffu, (i >> 5) == window ? page_cur : page_nxt, i & 31);
    };
    __syncthreads();  // barriers initialised
    const uint64_t pol = l2_evict_first_policy();
    auto issue = [&](int i) {
        const int tile = first + TR_WARPS * i;
        const int32_t pg = page_of(i);
        if (lane != 0) return;
        const int s = i % TR_STAGES;
        uint64_t* bar = &S.bar[warp][s];
        if (pg < 0) {
            mbar_arrive_expect_tx(bar, 0);  // completes the phase with no data
            return;
        }
        const int sub = tile % subs;
        const size_t so = scale_sub_off(pg, h, nkv, kv_bs, sub);
        mbar_arrive_expect_tx(bar, STAGE_BYTES);
        bulk_g2s(S.k[warp][s], P.cache.k + kv_sub_off(pg, h, nkv, kv_bs, sub), SUB_K_BYTES, bar,
                 pol);
        tma_load_3d(S.v[warp][s], &P.vmap, 0, sub * TILE, (int)page_head(pg, h, nkv), bar, pol);
        bulk_g2s(S.sc[warp][s][0], P.cache.kscale + so, SUB_S_BYTES, bar, pol);
        bulk_g2s(S.sc[warp][s][1], P.cache.vscale + so, SUB_S_BYTES, bar, pol);
    };
    for (int i = 0; i < TR_STAGES && i < mine; i++) issue(i);

    // ---- Q's codes while the first copies are in flight (article 9-2 §2 seg. 1)
    // A warp's rows, their loads in flight together: a chunk pays this prologue before it
    // can use its first tile.
    constexpr int QROWS = TR_ROWS / TR_WARPS;
    float4 qx[QROWS];
    load_type<HILO>(P.dtype, [&](auto type) {
#pragma unroll
        for (int i = 0; i < QROWS; i++) {
            const int r = warp + i * TR_WARPS, rr = rt * TR_ROWS + r, node = rr / G;
            qx[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (r < rows)
                qx[i] = load_q4(P.q, decltype(type)::value, (int64_t)(q0 + node) * P.q_st +
                                                                (h * G + rr % G) * P.q_sh + 4 * lane);
        }
    });
#pragma unroll
    for (int i = 0; i < QROWS; i++) {
        const int r = warp + i * TR_WARPS;
        float qs;
        const uint32_t u = quantize_q_lane(qx[i], qs) ^ 0x80808080u;
        // this lane's codes are elements 8c + 4s .. + 3 of block lane / 8, c = lane % 8 / 2,
        // s = lane % 2: registers half and half + 2 of k-step s for lane (row % 8, c)
        uint32_t* f = reinterpret_cast<uint32_t*>(
            &S.qf[r >> 4][lane >> 3][lane & 1][(r & 7) * 4 + ((lane & 7) >> 1)]);
        f[(r >> 3) & 1] = hsub2(__byte_perm(u, 0x64646464u, 0x4140), 0x64806480u);
        f[((r >> 3) & 1) + 2] = hsub2(__byte_perm(u, 0x64646464u, 0x4342), 0x64806480u);
        if ((lane & 7) == 0) S.qsc[r][lane >> 3] = qs;
    }
    __syncthreads();

    // Row half of 16-row tile mt is 16 mt + gq + 8 half.  Per row: running max (base
    // 2), partial sum over this lane's tokens, and O: D[mt][cg][0] elements 16cg + 2j,
    // D[mt][cg][1] 16cg + 2j + 1 (column j)
    float M[MT][2], sum[MT][2];
    float D[MT][HD / 16][2][4];
    // a row's weights go to the matrix instructions scaled by 2^-ev; per row, so that
    // what a row does not see cannot cost it precision
    int ev[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
#pragma unroll
        for (int half = 0; half < 2; half++) {
            M[mt][half] = M_INIT;
            sum[mt][half] = 0.0f;
            ev[mt][half] = -126;
        }
#pragma unroll
        for (int cg = 0; cg < HD / 16; cg++)
#pragma unroll
            for (int j = 0; j < 4; j++) D[mt][cg][0][j] = D[mt][cg][1][j] = 0.0f;
    }
    const float kmul = inv127() * P.scale * TR_LOG2E;
    auto scale_row = [&](int mt, int half, float f) {
#pragma unroll
        for (int cg = 0; cg < HD / 16; cg++)
#pragma unroll
            for (int j = 0; j < 2; j++) {
                D[mt][cg][j][2 * half] *= f;
                D[mt][cg][j][2 * half + 1] *= f;
            }
    };

    auto step = [&](int st, int tile, auto masked_c) {
        constexpr bool MASKED = decltype(masked_c)::value;
        // lane = token: its score multiplier and V step.  A token past the end gets
        // 0 for both: what its row of the page holds must not matter.
        const bool live = !MASKED || tile * TILE + lane < n;
        const float vstep = live ? __fmul_rn(S.sc[warp][st][1][lane], inv127()) : 0.0f;
        S.mul[warp][0][lane] = live ? __fmul_rn(S.sc[warp][st][0][lane], kmul) : 0.0f;
        S.mul[warp][1][lane] = vstep;
        auto bits = [](float x) -> uint32_t {  // of a finite |x|, else 0
            const uint32_t u = __float_as_uint(x) & 0x7FFFFFFFu;
            return u < 0x7F800000u ? u : 0u;
        };
        const uint32_t vtop = MASKED ? 0u : __reduce_max_sync(0xffffffffu, bits(vstep));
        __syncwarp();
        // ---- scores: s[mt][i][half] = (token 8c + r_i, token 8c + 4 + r_i), r_i = (i + c) % 4
        float2 s[MT][4][2];
#pragma unroll
        for (int bb = 0; bb < NB; bb++) {
            uint2 w[4];
#pragma unroll
            for (int i = 0; i < 4; i++)
                w[i] = *reinterpret_cast<const uint2*>(
                    S.k[warp][st] + 1024 * bb + (8 * ((i + (gq >> 1)) & 3) + gq) * 32 + 8 * c4);
            float d[MT][4][4];
#pragma unroll
            for (int ks = 0; ks < 2; ks++) {
                uint32_t qa[MT][4];
#pragma unroll
                for (int mt = 0; mt < MT; mt++) {
                    const uint4 f = S.qf[mt][bb][ks][lane];
                    qa[mt][0] = f.x;
                    qa[mt][1] = f.y;
                    qa[mt][2] = f.z;
                    qa[mt][3] = f.w;
                }
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const uint32_t u = (ks ? w[i].y : w[i].x) ^ 0x80808080u;
                    const uint32_t b0 = hsub2(__byte_perm(u, 0x64646464u, 0x4140), 0x64806480u);
                    const uint32_t b1 = hsub2(__byte_perm(u, 0x64646464u, 0x4342), 0x64806480u);
#pragma unroll
                    for (int mt = 0; mt < MT; mt++) {
                        if (ks == 0) d[mt][i][0] = d[mt][i][1] = d[mt][i][2] = d[mt][i][3] = 0.0f;
                        mma_f16_16816(d[mt][i], qa[mt], b0, b1);
                    }
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int half = 0; half < 2; half++) {
                    const float qs = S.qsc[16 * mt + gq + 8 * half][bb];
                    const float2 q2 = make_float2(qs, qs);
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const float2 dv = make_float2(d[mt][i][2 * half], d[mt][i][2 * half + 1]);
                        s[mt][i][half] = bb == 0 ? __fmul2_rn(dv, q2) : __ffma2_rn(dv, q2, s[mt][i][half]);
                    }
                }
        }
        uint32_t win[MT][2];  // visible tokens of the rows
        bool grow = false;
        {
            float2 km[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int t = 8 * c4 + ((i + c4) & 3);
                km[i] = make_float2(S.mul[warp][0][t], S.mul[warp][0][t + 4]);
            }
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int half = 0; half < 2; half++) {
                    if (MASKED) {
                        const int r = 16 * mt + gq + 8 * half;
                        win[mt][half] = r < rows ? node_window(P, q0, (rt * TR_ROWS + r) / G, nb,
                                                               tile * TILE - base)
                                                 : 0u;
                    }
                    float top = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        float2& x = s[mt][i][half];
                        x = __fmul2_rn(x, km[i]);
                        if (MASKED) {
                            const int t = 8 * c4 + ((i + c4) & 3);
                            x.x = (win[mt][half] >> t) & 1u ? x.x : -INFINITY;
                            x.y = (win[mt][half] >> (t + 4)) & 1u ? x.y : -INFINITY;
                        }
                        top = fmaxf(top, fmaxf(x.x, x.y));
                    }
                    grow |= top > M[mt][half] + TR_SLACK;
                }
        }
        if (__any_sync(0xffffffffu, grow)) {
            // rare: some row's maximum grew by a wide margin -> rescale its state
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int half = 0; half < 2; half++) {
                    float m = M[mt][half];
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        m = fmaxf(m, fmaxf(s[mt][i][half].x, s[mt][i][half].y));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                    const float f = tr_ex2(M[mt][half] - m);
                    M[mt][half] = m;
                    sum[mt][half] *= f;
                    scale_row(mt, half, f);
                }
        }
        // ---- weights.  ev keeps the largest V step that the row sees times 2^-ev below
        // 2^7, so with p <= 2^8 a weight stays below 2^15, inside the fp16 range; a tile
        // that needs a larger ev first scales the row of O by the exact power of two
        // 2^(old - new).  A step that is not finite does not count: its row is lost where
        // it is seen.
        float2 vm[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int t = 8 * c4 + ((i + c4) & 3);
            vm[i] = make_float2(S.mul[warp][1][t], S.mul[warp][1][t + 4]);
        }
        bool wide = false;
        int en[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; mt++)
#pragma unroll
            for (int half = 0; half < 2; half++) {
                uint32_t vb = vtop;
                if (MASKED) {
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int t = 8 * c4 + ((i + c4) & 3);
                        if ((win[mt][half] >> t) & 1u) vb = max(vb, bits(vm[i].x));
                        if ((win[mt][half] >> (t + 4)) & 1u) vb = max(vb, bits(vm[i].y));
                    }
                    vb = max(vb, __shfl_xor_sync(0xffffffffu, vb, 1));
                    vb = max(vb, __shfl_xor_sync(0xffffffffu, vb, 2));
                }
                en[mt][half] = max(ev[mt][half], (int)(vb >> 23) - 133);
                wide |= en[mt][half] != ev[mt][half];
            }
        if (__any_sync(0xffffffffu, wide)) {
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int half = 0; half < 2; half++) {
                    const int by = ev[mt][half] - en[mt][half];
                    scale_row(mt, half, by >= -126 ? pow2i(by) : 0.0f);
                    ev[mt][half] = en[mt][half];
                }
        }
        // token pair i of row half -> A register (half + 2 (i % 2)) of k-step i / 2
        uint32_t hi[MT][2][4], lo[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; mt++)
#pragma unroll
            for (int half = 0; half < 2; half++) {
                const float vsc = pow2i(-ev[mt][half]);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float2 y = __fadd2_rn(s[mt][i][half],
                                                make_float2(-M[mt][half], -M[mt][half]));
                    const float2 p = make_float2(tr_ex2(y.x), tr_ex2(y.y));
                    sum[mt][half] += p.x + p.y;
                    float2 w = __fmul2_rn(p, __fmul2_rn(vm[i], make_float2(vsc, vsc)));
                    if (MASKED) {  // a masked token's V step may be anything
                        const int t = 8 * c4 + ((i + c4) & 3);
                        w.x = (win[mt][half] >> t) & 1u ? w.x : 0.0f;
                        w.y = (win[mt][half] >> (t + 4)) & 1u ? w.y : 0.0f;
                    }
                    const uint32_t wh = f2_to_h2(w.x, w.y);
                    hi[mt][i >> 1][half + 2 * (i & 1)] = wh;
                    if (HILO) {
                        const float2 back = h2_to_f2(wh);
                        lo[mt][i >> 1][half + 2 * (i & 1)] = f2_to_h2(w.x - back.x, w.y - back.y);
                    }
                }
            }
        // ---- values: lane L gives the V row tok(L / 8, L % 8) of each 16-byte chunk
        const int tv = 4 * (lane & 7) + (((lane >> 3) + ((lane & 7) >> 1)) & 3);
        const uint32_t vrow = smem_u32(S.v[warp][st]) + (uint32_t)tv * HD;
#pragma unroll
        for (int cg = 0; cg < HD / 16; cg++) {
            uint32_t r[4];
            ldsm_x4_trans(vrow + ((uint32_t)(cg ^ (tv & 7)) << 4), r[0], r[1], r[2], r[3]);
            uint32_t be[4], bo[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint32_t u = r[j] ^ 0x80808080u;
                be[j] = hsub2(__byte_perm(u, 0x64646464u, 0x4240), 0x64806480u);
                bo[j] = hsub2(__byte_perm(u, 0x64646464u, 0x4341), 0x64806480u);
            }
#pragma unroll
            for (int ks = 0; ks < 2; ks++)
#pragma unroll
                for (int mt = 0; mt < MT; mt++) {
                    mma_f16_16816(D[mt][cg][0], hi[mt][ks], be[2 * ks], be[2 * ks + 1]);
                    mma_f16_16816(D[mt][cg][1], hi[mt][ks], bo[2 * ks], bo[2 * ks + 1]);
                    if (HILO) {
                        mma_f16_16816(D[mt][cg][0], lo[mt][ks], be[2 * ks], be[2 * ks + 1]);
                        mma_f16_16816(D[mt][cg][1], lo[mt][ks], bo[2 * ks], bo[2 * ks + 1]);
                    }
                }
        }
    };

    bool failed = false;
    for (int i = 0; i < mine; i++) {
        const int st = i % TR_STAGES, tile = first + TR_WARPS * i;
        if ((i >> 5) != window) {
            window = i >> 5;
            page_cur = page_nxt;
            page_nxt = load_window(window + 1);
        }
        const int32_t pg = page_of(i);
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&S.bar[warp][st], (i / TR_STAGES) & 1))) {
            // let the copies in flight land before leaving (bounded)
            for (int j = i; j < mine && j < i + TR_STAGES; j++)
                __all_sync(0xffffffffu, mbar_wait_bounded(&S.bar[warp][j % TR_STAGES],
                                                          (j / TR_STAGES) & 1));
            if (lane == 0) atomicOr(P.status, KQ8_STATUS_TIMEOUT);
            failed = true;
            break;
        }
        if (pg >= 0) {
            if ((tile + 1) * TILE <= base)
                step(st, tile, std::false_type{});
            else
                step(st, tile, std::true_type{});
        }
        __syncwarp();
        if (i + TR_STAGES < mine) issue(i + TR_STAGES);
    }

    // ---- merge the warps (the rings become [warp][rows][HD] accumulators)
    const bool cta_failed = __syncthreads_or(failed ? 1 : 0) != 0;
    float* macc = reinterpret_cast<float*>(S.v);
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
        for (int half = 0; half < 2; half++) {
            float t = sum[mt][half];
            t += __shfl_xor_sync(0xffffffffu, t, 1);
            t += __shfl_xor_sync(0xffffffffu, t, 2);
            const float f = pow2i(ev[mt][half]);
            const int r = 16 * mt + gq + 8 * half;
            float* row = macc + (warp * TR_ROWS + r) * HD;
#pragma unroll
            for (int cg = 0; cg < HD / 16; cg++)
                *reinterpret_cast<float4*>(row + 16 * cg + 4 * c4) =
                    make_float4(D[mt][cg][0][2 * half] * f, D[mt][cg][1][2 * half] * f,
                                D[mt][cg][0][2 * half + 1] * f, D[mt][cg][1][2 * half + 1] * f);
            if (c4 == 0) S.ms[warp][r] = make_float2(M[mt][half], t);
        }
    __syncthreads();
    const size_t pair = ((size_t)blockIdx.z * nkv + h) * P.row_tiles + rt;
    auto out_at = [&](int r) -> size_t {
        const int rr = rt * TR_ROWS + r;
        return ((size_t)(q0 + rr / G) * P.nq + (size_t)h * G + rr % G) * HD + 4 * lane;
    };
    for (int r = warp; r < rows; r += TR_WARPS) {
        float m = M_INIT, den = 0.0f;
#pragma unroll
        for (int w = 0; w < TR_WARPS; w++) m = fmaxf(m, S.ms[w][r].x);
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < TR_WARPS; w++) {
            const float2 ms = S.ms[w][r];
            const float f = tr_ex2(ms.x - m);
            const float4 x = reinterpret_cast<const float4*>(macc + (w * TR_ROWS + r) * HD)[lane];
            den += ms.y * f;
            a.x += x.x * f;
            a.y += x.y * f;
            a.z += x.z * f;
            a.w += x.w * f;
        }
        if (nch > 1) {
            const size_t pr = (pair * TR_ROWS + r) * P.num_chunks + chunk;
            reinterpret_cast<float4*>(P.part_acc + pr * HD)[lane] = a;
            if (lane == 0) P.part_ms[pr] = make_float2(m, cta_failed ? -1.0f : den);
        } else if (!cta_failed) {  // a row that sees no token gives 0
            const float inv = den == 0.0f ? 0.0f : 1.0f;
            const float dv = den == 0.0f ? 1.0f : den;
            store_out4(P.out, P.dtype, out_at(r),
                       make_float4(a.x / dv * inv, a.y / dv * inv, a.z / dv * inv, a.w / dv * inv));
        }
    }
    if (nch == 1) return;

    // ---- the last CTA of this (sequence, KV head, row tile) merges the chunks
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        S.last = atomicAdd(&P.counters[pair], 1u) == (unsigned)(nch - 1);
    }
    __syncthreads();
    if (!S.last) return;
    __threadfence();
    for (int r = warp; r < rows; r += TR_WARPS) {
        const size_t at = (pair * TR_ROWS + r) * P.num_chunks;
        float m = M_INIT, den = 0.0f;
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        bool bad = false;
#pragma unroll 8
        for (int c = 0; c < nch; c++) {
            const float2 ms = __ldcg(&P.part_ms[at + c]);
            const float4 x =
                __ldcg(reinterpret_cast<const float4*>(P.part_acc + (at + c) * HD) + lane);
            bad |= ms.y < 0.0f;
            const float mn = fmaxf(m, ms.x);
            const float fo = tr_ex2(m - mn), fn = tr_ex2(ms.x - mn);
            den = den * fo + ms.y * fn;
            a.x = a.x * fo + x.x * fn;
            a.y = a.y * fo + x.y * fn;
            a.z = a.z * fo + x.z * fn;
            a.w = a.w * fo + x.w * fn;
            m = mn;
        }
        if (bad) continue;  // a timed-out chunk: the row stays as it was
        const float inv = den == 0.0f ? 0.0f : 1.0f;
        const float dv = den == 0.0f ? 1.0f : den;
        store_out4(P.out, P.dtype, out_at(r),
                   make_float4(a.x / dv * inv, a.y / dv * inv, a.z / dv * inv, a.w / dv * inv));
    }
    if (threadIdx.x == 0) P.counters[pair] = 0;  // ready for the next call
}

// A call's split: rows of a tile, sequences per launch (so that the tickets of a
// launch fit the header's counters), row tiles, chunks and the partials' places.
struct TreePlan {
    int tile_rows = 16;  // 16, 32: kq8_tree_kernel; 128, 256: the tensor cores
    int ctas = 0;        // of the tensor cores' kernel
    int seqs = 0, row_tiles = 1, chunk_tiles = TR_WARPS, num_chunks = 1;
    size_t off_ms = 0, off_acc = 0, off_spill = 0, total = TR_HEADER;
};
constexpr int64_t TR_PARTS = 512ll << 20;  // bytes of partials a call may take

// Sub-tiles per chunk, at most TR_MAX_CHUNK (a long chunk of a ragged batch is a long
// tail): of the chunk counts that allow, the one whose waves of resident CTAs take
// least, a CTA's prologue and merge costing TR_CTA_TILES sub-tiles of a warp beside its
// walk.  Uniform lists of 512 sub-tiles, 128 of them, 32 rows: 184 us with a CTA's
// cost put at 5 sub-tiles, 174 at 10; ragged lists of 1K to 32K tokens, 512 of them: chunks
// of at most 64 sub-tiles 719 us, 96 695, 128 658, 192 657.
constexpr int64_t TR_CTA_TILES = 10;
int64_t tree_chunk(int64_t pairs, int64_t tiles, int ctas_per_sm) {
    const int64_t slots = (int64_t)device_sms() * ctas_per_sm;
    const int64_t least = (tiles + TR_MAX_CHUNK - 1) / TR_MAX_CHUNK;
    int64_t best = TR_WARPS, cost = INT64_MAX;
    for (int64_t k = least > 1 ? least : 1; k <= 4 * least + 16; k++) {
        const int64_t c = ((tiles + k - 1) / k + TR_WARPS - 1) / TR_WARPS * TR_WARPS;
        if (c < TR_WARPS) break;
        const int64_t waves = (pairs * ((tiles + c - 1) / c) + slots - 1) / slots;
        if (waves * (c / TR_WARPS + TR_CTA_TILES) < cost) {
            cost = waves * (c / TR_WARPS + TR_CTA_TILES);
            best = c;
        }
        if (c == TR_WARPS) break;
    }
    return best;
}

// Rows of a tile.  16 x 16384 tokens, 8 KV heads, bf16 (fp32): 16 rows take 104 (116) us
// on one 16-row tile a warp; 32 rows 174 (210) on two, and on a tensor-core tile of 128
// rows, which costs 64 rows as much, 226 (332); two tiles of 32 rows take twice 174, so
// from 33 rows on it is the tensor cores: 128 rows 234 (339), 256 rows 340 on a pair of
// tiles that share K and V, twice 234 as lists of one tile.
TreePlan tree_plan(int B, int nq, int nkv, int max_seq_len, int max_q_len, bool hilo) {
    TreePlan p;
    const int64_t rows = (int64_t)max_q_len * (nq / nkv);
    p.tile_rows = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 128 || hilo ? 128 : 256;
    p.row_tiles = (int)((rows + p.tile_rows - 1) / p.tile_rows);
    if (p.row_tiles < 1) p.row_tiles = 1;
    const int64_t per_seq = (int64_t)nkv * p.row_tiles;
    const int64_t tiles = ((int64_t)max_seq_len + TILE - 1) / TILE;
    const int64_t part = (int64_t)p.tile_rows * (HD * sizeof(float) + sizeof(float2));
    size_t parts = 0;
    if (p.tile_rows <= 32) {
        if (per_seq > (int64_t)TR_COUNTERS) return p;  // seqs = 0: unsupported
        p.seqs = (int)((int64_t)TR_COUNTERS / per_seq);
        if (p.seqs > B) p.seqs = B;
        const int64_t pairs = (int64_t)p.seqs * per_seq;
        int64_t c =
            tree_chunk(pairs, tiles, p.tile_rows == 16 ? TreeShape<1>::CTAS : TreeShape<2>::CTAS);
        while (c < tiles && pairs * ((tiles + c - 1) / c) * part > TR_PARTS) c *= 2;
        p.chunk_tiles = (int)c;
        p.num_chunks = tiles > 0 ? (int)((tiles + c - 1) / c) : 1;
        if (p.num_chunks > 1) parts = (size_t)(pairs * p.tile_rows * p.num_chunks);
    } else {
        // one CTA per SM, at least two steps each; two parts a CTA
        p.seqs = B;
        const int64_t steps = (tiles + 3) / 4 * per_seq * B;
        p.ctas = device_sms();
        if ((steps + 1) / 2 < p.ctas) p.ctas = steps > 1 ? (int)((steps + 1) / 2) : 1;
        parts = (size_t)p.ctas * 2 * p.tile_rows;
    }
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    p.off_ms = TR_HEADER;
    p.off_acc = up(p.off_ms + parts * sizeof(float2));
    p.off_spill = up(p.off_acc + parts * HD * sizeof(float));
    p.total = p.off_spill + (hilo ? (size_t)p.ctas * 2 * HD * 128 * sizeof(float) : 0);
    return p;
}

template <int MT, bool HILO>
int launch_tree(const TreeParams& p, dim3 grid, cudaStream_t s) {
    static std::atomic<uint64_t> opted{0};
    return launch_smem(kq8_tree_kernel<MT, HILO>, opted, grid, TR_THREADS,
                       sizeof(TreeSmem<MT>) + 1024,  // slack to round the base up
                       s, p);
}

}  // namespace
}  // namespace kq8

using namespace kq8;

extern "C" {

size_t kq8_tree_workspace_bytes(int32_t B, int32_t nq, int32_t nkv, int32_t max_seq_len,
                                int32_t max_q_len) {
    if (B < 0 || nq < 1 || nkv < 1 || nq % nkv || max_seq_len < 0 || max_q_len < 0) return 0;
    const size_t a = tree_plan(B, nq, nkv, max_seq_len, max_q_len, false).total;
    const size_t b = tree_plan(B, nq, nkv, max_seq_len, max_q_len, true).total;
    return a > b ? a : b;
}

int kq8_tree_attn(void* out, const void* q, int32_t dtype, size_t q_token_stride,
                  size_t q_head_stride, int32_t total_q, const kq8_cache_t* cache,
                  const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens,
                  const int32_t* q_offsets, const uint32_t* tree_mask, int32_t mask_words,
                  int32_t max_seq_len, int32_t max_q_len, int32_t B, int32_t nq, float scale,
                  void* workspace, size_t workspace_bytes, kq8_stream_t stream) {
    int rc = check_cache_args(cache);
    if (rc) return rc;
    if (dtype != KQ8_F32 && dtype != KQ8_F16 && dtype != KQ8_BF16) return KQ8_ERR_UNSUPPORTED;
    if (B < 0 || nq < 1 || total_q < 0 || max_seq_len < 0 || max_q_len < 0 || max_pages < 0 ||
        mask_words < 0)
        return KQ8_ERR_INVALID_ARG;
    const int nkv = cache->num_kv_heads;
    if (nq % nkv != 0 || nq / nkv > MAX_G) return KQ8_ERR_UNSUPPORTED;
    if ((int64_t)max_seq_len > (int64_t)max_pages * cache->kv_bs) return KQ8_ERR_INVALID_ARG;
    if (max_q_len > max_seq_len) return KQ8_ERR_INVALID_ARG;
    if (max_seq_len >= (1 << 29) || B > 65535 || nkv > 65535 || max_q_len > KQ8_TREE_MAX_NODES)
        return KQ8_ERR_UNSUPPORTED;
    if (tree_mask && (int64_t)mask_words * 32 < max_q_len) return KQ8_ERR_INVALID_ARG;
    const TreePlan plan = tree_plan(B, nq, nkv, max_seq_len, max_q_len, dtype != KQ8_BF16);
    if (!workspace || (uintptr_t)workspace % 256 != 0 || workspace_bytes < plan.total)
        return KQ8_ERR_WORKSPACE;
    if (B == 0 || max_q_len == 0) return KQ8_OK;
    if (plan.seqs < 1) return KQ8_ERR_UNSUPPORTED;
    if (!out || !q || !seq_lens || !q_offsets || !page_table) return KQ8_ERR_INVALID_ARG;
    // a lane reads 4 elements of a q row and writes 4 of an output row
    const size_t quad = dtype == KQ8_F32 ? 16 : 8;
    if ((uintptr_t)out % quad || (uintptr_t)q % quad || q_token_stride % 4 || q_head_stride % 4 ||
        q_token_stride > MAX_STRIDE || q_head_stride > MAX_STRIDE ||
        (tree_mask && (uintptr_t)tree_mask % 4))
        return KQ8_ERR_INVALID_ARG;
    // q is read while other rows are written
    if (stretches_meet(out, rows_bytes(total_q, (size_t)nq * HD, nq, HD, quad / 4), q,
                       rows_bytes(total_q, q_token_stride, nq, q_head_stride, quad / 4)))
        return KQ8_ERR_INVALID_ARG;
    TreeParams p;
    std::memset(&p, 0, sizeof(p));
    rc = encode_vmap(&p.vmap, *cache, false);
    if (rc) return rc;
    p.out = out;
    p.q = q;
    p.q_st = (int64_t)q_token_stride;
    p.q_sh = (int64_t)q_head_stride;
    p.dtype = dtype;
    p.total_q = total_q;
    p.cache = *cache;
    p.page_table = page_table;
    p.max_pages = max_pages;
    p.seq_lens = seq_lens;
    p.q_off = q_offsets;
    p.mask = tree_mask;
    p.mask_words = mask_words;
    p.max_seq_len = max_seq_len;
    p.max_q_len = max_q_len;
    p.nq = nq;
    p.G = nq / nkv;
    p.scale = scale;
    p.chunk_tiles = plan.chunk_tiles;
    p.num_chunks = plan.num_chunks;
    p.row_tiles = plan.row_tiles;
    char* ws = static_cast<char*>(workspace);
    p.part_ms = reinterpret_cast<float2*>(ws + plan.off_ms);
    p.part_acc = reinterpret_cast<float*>(ws + plan.off_acc);
    p.spill = reinterpret_cast<float*>(ws + plan.off_spill);
    p.status = reinterpret_cast<uint32_t*>(ws);
    p.counters = reinterpret_cast<uint32_t*>(ws + TR_STATUS_BYTES);
    const cudaStream_t st = (cudaStream_t)stream;
    const bool hilo = dtype != KQ8_BF16;
    for (p.b0 = 0; p.b0 < B; p.b0 += plan.seqs) {
        const int seqs = B - p.b0 < plan.seqs ? B - p.b0 : plan.seqs;
        const dim3 grid((unsigned)(plan.num_chunks * plan.row_tiles), (unsigned)nkv, (unsigned)seqs);
        p.seqs = seqs;
        if (plan.ctas)
            rc = launch_tree_tc(p, plan.tile_rows, plan.ctas, st);
        else if (plan.tile_rows == 16)
            rc = hilo ? launch_tree<1, true>(p, grid, st) : launch_tree<1, false>(p, grid, st);
        else
            rc = hilo ? launch_tree<2, true>(p, grid, st) : launch_tree<2, false>(p, grid, st);
        if (rc) return rc;
    }
    return KQ8_OK;
}

}  // extern "C"
