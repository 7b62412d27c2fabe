// kq8_prompt.cu -- causal attention over packed prompts from their own fp16 / bf16
// queries, keys and values (a prompt's first pass, before or beside its write to
// the cache), on the 5th-generation tensor cores.
//
//   o_i = sum_{j <= i} softmax_j(scale * q_i . k_j) v_j   within each sequence,
// query head h reading KV head h / G.
//
// Work decomposition.  A CTA (one per SM: all 512 TMEM columns) takes two query
// tiles A and B of 128 rows of one KV head -- 128 / G consecutive tokens x its G
// query heads each -- and walks the sequence in blocks of 128 tokens up to its
// last row.  The rows share every K and V block, and TMA brings a tile's rows in
// with one box {64 elements, G heads, 128 / G tokens} per half row.
// Roles (three warpgroups, which meet on mbarriers only):
//   warps 0-3, 4-7  softmax of tile A, B, one thread per row (TMEM lane): the 128
//                   scores of a block in registers, the running maximum and sum in
//                   fp32, the weights p = 2^(x - m) back to TMEM as 16-bit pairs; O is
//                   rescaled in place only when the maximum grows by more than 2^8;
//   warp 8          one lane issues S = Q_t K^T, the tiles in turn (8 MMAs of M = N =
//                   128, K = 16, both operands in shared memory);
//   warps 9, 11     one lane each issues O_t += P_t V of tile A, B (A in TMEM, V read
//                   with the dimension as its major axis, so that the rows are used as
//                   they lie in memory);
//   warp 10         TMA loads: Q once, then K and V blocks through a ring of five; at
//                   the end it clears the rows of the last V block that lie behind the
//                   sequence.
// TMEM holds O of both tiles (2 x 128 columns), the weights of both (2 x 64) and one
// block of scores (128) that the tiles use in turn: a row's scores are in registers a
// few hundred cycles after their product, so the next product of the other tile, and
// then the tile's own next one, run beside the softmax instead of behind it.  (With
// the weights over their own scores, and so S_t(j+1) behind PV_t(j), a step took 3780
// cycles against 2048 of MMAs.)
// What bounds it: 16 MMAs of 128 x 128 x 16 per tile and block, 8192 FLOP per cycle and
// SM at best (64 cycles each, measured), against 16384 exponentials per tile in the
// same time (4 cycles a warp and sub-partition, measured).
// Measured, bf16: four prompts of 1000 to 8192 tokens, 32/8 heads, 870 us = 1.34 PFLOP/s
// (0.68 of a library GEMM's burst rate; the tensor pipe is active in 65 % of an SM's
// cycles, the rest is the hand-over between softmax and MMA threads and a CTA's first and
// last block); 4059 tokens, 16/8 heads, 56 us: 256 CTAs of 1 to 32 blocks on 152 SMs,
// longest first; 506 tokens 12 us, four blocks one after the other.
#include <cstdint>
#include <cstring>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kq8_internal.h"
#include "kq8_tc.cuh"

namespace kq8 {
namespace {

constexpr int PR_ROWS = 128;   // rows per query tile
constexpr int PR_BLK = 128;    // tokens per block
constexpr int PR_RING = 5;     // K / V blocks in shared memory
constexpr int PR_THREADS = 12 * 32;
constexpr int PR_S_WARP = 8, PR_PVA_WARP = 9, PR_LOAD_WARP = 10, PR_PVB_WARP = 11;
// registers per thread: 168 at launch; the softmax warpgroups take what the
// third one gives back (2 * 216 + 72 = 3 * 168)
constexpr int PR_REGS_SOFTMAX = 216, PR_REGS_REST = 72;
constexpr uint32_t PR_PANEL = PR_ROWS * 128;   // 128 rows x 64 16-bit elements
constexpr uint32_t PR_TILE = 2 * PR_PANEL;     // 128 rows x 128 elements
// TMEM columns: O_t at 128 t, S at 256, P_t at 384 + 64 t
constexpr uint32_t PR_COLS = 512, PR_COL_S = 256, PR_COL_P = 384;
// shared memory: Q tiles, ring, barriers
constexpr uint32_t PR_SM_Q = 0, PR_SM_RING = 2 * PR_TILE;
constexpr uint32_t PR_SM_BAR = PR_SM_RING + PR_RING * PR_TILE;
constexpr uint32_t PR_SM_TMEM = PR_SM_BAR + 256, PR_SM_ABORT = PR_SM_TMEM + 4;
constexpr uint32_t PR_SMEM = PR_SM_ABORT + 4 + 1024;  // slack to round the base up to 1 KB
static_assert(PR_SMEM <= 232448, "shared memory of one CTA");

constexpr int PB_Q = 0;          // Q has landed
// The ring's length is odd, so K(j) takes the place of V(j-3), and V(j) that of K(j-2).
// The S thread waits for K's phases of a place only, the PV threads for V's; a parity
// wait is sound as the phase in between has completed by then: before S(j) the tiles
// have read S(j-1), so they had finished P(j-2), for which PV(j-3) was done; before
// PV(j) a PV thread has seen P(j-1), which came of S(j-1) behind S(j-2).
constexpr int PB_FULL = 1;       // [ring] block has landed
constexpr int PB_EMPTY = 6;      // [ring] both tiles have used the block
constexpr int PB_S = 11;         // [tile] commit after S of the tile
constexpr int PB_SR = 13;        // 4 softmax warps hold S in registers (the tiles in turn)
constexpr int PB_P = 14;         // [tile][half] 4 softmax warps wrote 64 columns of P_t
                                 // (and, before the first half, rescaled O_t)
constexpr int PB_PV = 18;        // [tile] commit after PV_t
constexpr int PB_LAST = 20;      // the last V has landed, where rows in it are to be cleared
constexpr int PB_TAIL = 21;      // and they are
constexpr int PB_FINAL = 22;     // [MMA thread] last commit, waited on before TMEM is freed
constexpr int PB_COUNT = 25;

constexpr float PR_LOG2E = 1.4426950408889634f;
constexpr float PR_SLACK = 8.0f;

struct PromptParams {
    CUtensorMap qmap, kmap, vmap;
    void* out;
    const int32_t* cu;
    int32_t total, max_len, nq, G;
    float scale;
    uint32_t* status;
};

__device__ __forceinline__ float pr_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        return f2_to_h2(lo, hi);
    }
}
__device__ __forceinline__ void pr_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

template <bool BF16>
__global__ void __launch_bounds__(PR_THREADS, 1)
    kq8_prompt_kernel(const __grid_constant__ PromptParams P) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = P.G, TQ = PR_ROWS / G;  // tokens per query tile
    // CTAs start in linear order: the (KV head, sequence) runs fastest and the
    // query tiles from the last, longest, to the first
    const unsigned lin = blockIdx.x + gridDim.x * (blockIdx.y + gridDim.y * blockIdx.z);
    const unsigned hbn = gridDim.y * gridDim.z;
    const int h = (int)((lin % hbn) % gridDim.y), b = (int)((lin % hbn) / gridDim.y);
    const int qt = (int)gridDim.x - 1 - (int)(lin / hbn);
    griddep_wait();
    griddep_launch_dependents();

    const int s0 = P.cu[b], L = P.cu[b + 1] - s0;
    if (s0 < 0 || L < 0 || L > P.max_len || (int64_t)s0 + L > P.total) {
        if (tid == 0 && qt == 0 && h == 0 && P.status) atomicOr(P.status, KQ8_STATUS_BAD_SEQLEN);
        return;
    }
    const int i0 = qt * 2 * TQ;  // first token of tile A; tile B follows
    if (i0 >= L) return;
    // blocks of the two tiles (tile B may be empty)
    const int lastA = min(i0 + TQ, L) - 1, lastB = min(i0 + 2 * TQ, L) - 1;
    const int nA = lastA / PR_BLK + 1;
    const int nB = i0 + TQ < L ? lastB / PR_BLK + 1 : 0;
    const int nblk = max(nA, nB);
    const bool tail = nblk * PR_BLK > L;  // the last block reaches behind the sequence

    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + PR_SM_BAR);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + PR_SM_TMEM);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + PR_SM_ABORT);
    if (warp == 0) {
        __syncwarp();
        tc::tmem_alloc(tslot, PR_COLS);
    }
    if (tid == 0) {
        for (int i = 0; i < PB_COUNT; i++) {
            uint32_t cnt = 1;
            // V is released by a PV thread per tile, K by the S thread, which arrives for
            // both: the ring's length is odd, so K and V take a place in turn
            if (i >= PB_EMPTY && i < PB_S) cnt = nB ? 2 : 1;
            if (i >= PB_SR && i < PB_PV) cnt = 4;
            mbar_init(bars + i, cnt);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tbase = *tslot;
    // A wait that runs out is recorded and makes every later wait that does not
    // succeed at once give up.
    auto wait = [&](int i, uint32_t parity) -> bool {
        if (mbar_try_wait(bars + i, parity)) return true;
        const long long t0 = clock64();
        while (!mbar_try_wait(bars + i, parity)) {
            if (*abort_flag) return false;
            if (clock64() - t0 > (1ll << 28)) {
                *abort_flag = 1;
                if (P.status) atomicOr(P.status, KQ8_STATUS_TIMEOUT);
                return false;
            }
        }
        return true;
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PR_REGS_REST));
        if (warp == PR_LOAD_WARP) {
            if (lane == 0) {
                // ---- loads: ring item 2 j is K of block j, 2 j + 1 its V
                const uint64_t pol = l2_evict_first_policy();
                const uint64_t keep = l2_evict_last_policy();
                const uint32_t qbytes = (uint32_t)(TQ * G) * 128u;
                mbar_arrive_expect_tx(bars + PB_Q, 2 * qbytes * (nB ? 2 : 1));
                for (int t = 0; t < (nB ? 2 : 1); t++)
                    for (int p = 0; p < 2; p++)
                        tma_load_3d(sm + PR_SM_Q + t * PR_TILE + p * PR_PANEL, &P.qmap, 64 * p, h * G,
                                    s0 + i0 + t * TQ, bars + PB_Q, pol);
                // the last V lands on a barrier of its own where the tail warp waits for it
                auto landed = [&](int it) {
                    return tail && it == 2 * nblk - 1 ? PB_LAST : PB_FULL + it % PR_RING;
                };
                int it = 0;
                for (; it < 2 * nblk; it++) {
                    const int s = it % PR_RING;
                    if (it >= PR_RING && !wait(PB_EMPTY + s, (it / PR_RING - 1) & 1)) break;
                    uint64_t* bar = bars + landed(it);
                    mbar_arrive_expect_tx(bar, PR_TILE);
                    for (int p = 0; p < 2; p++)
                        tma_load_3d(sm + PR_SM_RING + s * PR_TILE + p * PR_PANEL,
                                    it & 1 ? &P.vmap : &P.kmap, 64 * p, h, s0 + (it >> 1) * PR_BLK, bar,
                                    keep);
                }
                // an aborted CTA lets the copies in flight land (bounded)
                if (*abort_flag) {
                    mbar_wait_bounded(bars + PB_Q, 0);
                    for (int i = it > PR_RING ? it - PR_RING : 0; i < it; i++)
                        mbar_wait_bounded(bars + landed(i), landed(i) == PB_LAST ? 0 : (i / PR_RING) & 1);
                }
            }
            __syncwarp();
            if (tail && __all_sync(0xffffffffu, wait(PB_LAST, 0))) {
                // rows behind the sequence's end belong to others: weights of 0 must not
                // meet what they hold
                uint8_t* v = sm + PR_SM_RING + ((2 * nblk - 1) % PR_RING) * PR_TILE;
                for (int c = (L - (nblk - 1) * PR_BLK) * 8 + lane; c < PR_BLK * 8; c += 32)
                    for (int p = 0; p < 2; p++)
                        *reinterpret_cast<uint4*>(v + p * PR_PANEL + c * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                tc::fence_smem_to_async();
                __syncwarp();
                if (lane == 0) pr_arrive(bars + PB_TAIL);
            }
        } else if (warp == PR_S_WARP && lane == 0) {
            // ---- S of both tiles, in turn.  Operand rows are 128 bytes, swizzled; a
            // K-major step of 16 elements is 32 bytes along the row.
            const uint64_t dq = tc::sdesc_sw128(smem_u32(sm + PR_SM_Q), 16, 1024);
            const uint64_t dk = tc::sdesc_sw128(smem_u32(sm + PR_SM_RING), 16, 1024);
            constexpr uint32_t IDS = tc::IDesc<128, PR_BLK, BF16>::value;
            bool ok = wait(PB_Q, 0);
            int place = 0;
            uint32_t phase = 0, read = 0;  // of K of block j; S blocks issued so far
            for (int j = 0; ok && j < nblk; j++) {
                const uint64_t k = dk + (uint64_t)(place * (PR_TILE >> 4));
                ok = wait(PB_FULL + place, phase);
                for (int t = 0; ok && t < 2; t++) {
                    if (j >= (t ? nB : nA)) continue;
                    // the scores before these are in registers
                    if (read > 0 && !(ok = wait(PB_SR, (read - 1) & 1))) break;
                    read++;
                    tc::fence_after_sync();
                    const uint64_t a = dq + (uint64_t)(t * (PR_TILE >> 4));
#pragma unroll
                    for (int kk = 0; kk < HD / 16; kk++) {
                        const uint64_t o = (kk >> 2) * (PR_PANEL >> 4) + (kk & 3) * 2;
                        tc::mma_f16(tbase + PR_COL_S, a + o, k + o, IDS, kk > 0);
                    }
                    tc::mma_commit(bars + PB_S + t);
                }
                // a ring place is released when a later load waits for it
                if (ok && 2 * j + PR_RING < 2 * nblk) {
                    tc::mma_commit(bars + PB_EMPTY + place);
                    if (nB) pr_arrive(bars + PB_EMPTY + place);
                }
                if ((place += 2) >= PR_RING) place -= PR_RING, phase ^= 1;
            }
            tc::mma_commit(bars + PB_FINAL);  // completes once every MMA above has (bounded)
            mbar_wait_bounded(bars + PB_FINAL, 0);
        } else if ((warp == PR_PVA_WARP || (warp == PR_PVB_WARP && nB)) && lane == 0) {
            // ---- PV of tile t.  V's step of 16 tokens is two groups of eight rows.
            const int t = warp == PR_PVB_WARP ? 1 : 0, nt = t ? nB : nA;
            const uint64_t dv = tc::sdesc_sw128(smem_u32(sm + PR_SM_RING), PR_PANEL, 1024);
            constexpr uint32_t IDO = tc::IDesc<128, HD, BF16>::value | tc::IDESC_B_MN;
            const uint32_t tO = tbase + 128 * t, tP = tbase + PR_COL_P + 64 * t;
            bool ok = true;
            int place = 1;
            uint32_t phase = 0;
            for (int j = 0; ok && j < nt; j++) {
                const uint64_t v = dv + (uint64_t)(place * (PR_TILE >> 4));
                ok = tail && j + 1 == nblk ? wait(PB_TAIL, 0) : wait(PB_FULL + place, phase);
                // the two halves of P as they come
#pragma unroll
                for (int half = 0; half < 2; half++) {
                    if (!(ok = ok && wait(PB_P + 2 * t + half, j & 1))) break;
                    tc::fence_after_sync();
#pragma unroll
                    for (int kk = 4 * half; kk < 4 * half + 4; kk++)
                        tc::mma_f16_ta(tO, tP + 8 * kk, v + (uint64_t)(kk * (2048 >> 4)), IDO,
                                       j > 0 || kk > 0);
                }
                if (!ok) break;
                tc::mma_commit(bars + PB_PV + t);
                // (tile B sees at most one block more than tile A, and no later load waits
                // for the places of the last two blocks)
                if (2 * j + 1 + PR_RING < 2 * nblk) tc::mma_commit(bars + PB_EMPTY + place);
                if ((place += 2) >= PR_RING) place -= PR_RING, phase ^= 1;
            }
            tc::mma_commit(bars + PB_FINAL + 1 + t);
            mbar_wait_bounded(bars + PB_FINAL + 1 + t, 0);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PR_REGS_SOFTMAX));
        const int t = warp >> 2, nt = t ? nB : nA;
        const int row = (warp & 3) * 32 + lane;
        const int tok = i0 + t * TQ + row / G;  // this row's token
        const bool valid = row < TQ * G && tok < L;
        const int first = i0 + t * TQ;          // the tile's first token
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tbase + PR_COL_S + lanes, tO = tbase + 128 * t + lanes;
        const uint32_t tP = tbase + PR_COL_P + 64 * t + lanes;
        const float sl2 = P.scale * PR_LOG2E;
        const float slack = PR_SLACK / sl2;
        float M = -INFINITY;  // reference of the weights, in units of raw scores
        float2 sum = make_float2(0.0f, 0.0f);
        bool ok = true;
        for (int j = 0; j < nt; j++) {
            ok = __all_sync(0xffffffffu, wait(PB_S + t, j & 1));
            if (!ok) break;
            tc::fence_after_sync();
            float x[PR_BLK];
            tc::tmem_ld_cols<PR_BLK>(tS, x);
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) pr_arrive(bars + PB_SR);
            if ((j + 1) * PR_BLK - 1 > first) {  // a diagonal block: token c sees 0 .. tok
                const int vis = tok - j * PR_BLK;  // last visible column
#pragma unroll
                for (int c = 0; c < PR_BLK; c++) x[c] = c <= vis ? x[c] : -INFINITY;
            }
            float m4[4] = {x[0], x[1], x[2], x[3]};  // four chains: the latency, not the issue
#pragma unroll
            for (int c = 4; c < PR_BLK; c += 8)
#pragma unroll
                for (int i = 0; i < 4; i++)
                    m4[i] = fmaxf(m4[i], c + 4 + i < PR_BLK ? fmaxf(x[c + i], x[c + 4 + i]) : x[c + i]);
            const float mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
            const bool need = mt > M + slack || j == 0;
            // PV_t of the block before has read P_t and is in O_t
            if (j > 0) {
                ok = __all_sync(0xffffffffu, wait(PB_PV + t, (j - 1) & 1));
                if (!ok) break;
                tc::fence_after_sync();
            }
            if (j > 0 && __any_sync(0xffffffffu, need)) {
                const float f = need ? pr_ex2((M - mt) * sl2) : 1.0f;
                sum = __fmul2_rn(sum, make_float2(f, f));
#pragma unroll 1
                for (int c = 0; c < HD / 32; c++) {
                    float o[32];
                    tc::tmem_ld32(tO + 32 * c, o);
#pragma unroll
                    for (int i = 0; i < 32; i++) o[i] *= f;
                    tc::tmem_st32(tO + 32 * c, o);
                }
            }
            if (need) M = mt;
            const float2 sc = make_float2(sl2, sl2), off = make_float2(-M * sl2, -M * sl2);
#pragma unroll
            for (int q = 0; q < PR_BLK / 64; q++) {
                float w[32];  // 32 columns of 16-bit pairs
#pragma unroll
                for (int c = 0; c < 32; c++) {
                    const float2 y =
                        __ffma2_rn(make_float2(x[64 * q + 2 * c], x[64 * q + 2 * c + 1]), sc, off);
                    const float2 p = make_float2(pr_ex2(y.x), pr_ex2(y.y));
                    sum = __fadd2_rn(sum, p);
                    w[c] = __uint_as_float(pack2<BF16>(p.x, p.y));
                }
                tc::tmem_st32(tP + 32 * q, w);
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) pr_arrive(bars + PB_P + 2 * t + q);
            }
        }
        // ---- output after the last PV_t
        if (nt > 0 && ok && __all_sync(0xffffffffu, wait(PB_PV + t, (nt - 1) & 1))) {
            tc::fence_after_sync();
            const float inv = __fdiv_rn(1.0f, sum.x + sum.y);
            uint4* dst = reinterpret_cast<uint4*>(
                static_cast<uint16_t*>(P.out) +
                ((size_t)(s0 + tok) * P.nq + (size_t)h * G + row % G) * HD);
#pragma unroll 1
            for (int c = 0; c < HD / 32; c++) {
                float o[32];
                tc::tmem_ld32(tO + 32 * c, o);
                if (valid) {
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        dst[4 * c + i] =
                            make_uint4(pack2<BF16>(o[8 * i] * inv, o[8 * i + 1] * inv),
                                       pack2<BF16>(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                       pack2<BF16>(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                                       pack2<BF16>(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
                }
            }
        }
    }
    // ---- teardown: every role has left its loop and the last commit has completed
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        __syncwarp();
        tc::fence_after_sync();
        tc::tmem_dealloc(tbase, PR_COLS);
    }
}

// {128 elements, heads, tokens} with the given element strides, boxes of 64
// elements (one 128-byte swizzled row), `heads_box` heads and `tokens_box` tokens.
int row_map(CUtensorMap* map, bool bf16, const void* base, int64_t tokens, int64_t heads,
            size_t st, size_t sh, uint32_t heads_box, uint32_t tokens_box) {
    // a dimension of one never steps: its stride only has to be a legal one
    const uint64_t dims[3] = {HD, (uint64_t)heads, (uint64_t)tokens};
    const uint64_t strides[2] = {heads > 1 ? sh * 2 : HD * 2, tokens > 1 ? st * 2 : HD * 2};
    const uint32_t box[3] = {64u, heads_box, tokens_box};
    return encode_tensor_map(
        map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
        const_cast<void*>(base), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <bool BF16>
int launch_prompt(const PromptParams& p, dim3 grid, cudaStream_t s) {
    static std::atomic<uint64_t> opted{0};
    return launch_smem(kq8_prompt_kernel<BF16>, opted, grid, PR_THREADS, PR_SMEM, s, p);
}

}  // namespace
}  // namespace kq8

using namespace kq8;

extern "C" int kq8_prompt_attn(void* out, const void* q, const void* k, const void* v,
                               int32_t dtype, size_t q_token_stride, size_t q_head_stride,
                               size_t k_token_stride, size_t k_head_stride, size_t v_token_stride,
                               size_t v_head_stride, const int32_t* cu_seqlens, int32_t total,
                               int32_t max_len, int32_t B, int32_t nq, int32_t nkv, float scale,
                               uint32_t* status, kq8_stream_t stream) {
    if (dtype != KQ8_F16 && dtype != KQ8_BF16) return KQ8_ERR_UNSUPPORTED;
    if (B < 0 || total < 0 || max_len < 0 || nq < 1 || nkv < 1) return KQ8_ERR_INVALID_ARG;
    if (!(scale > 0.0f) || scale > 3.0e38f) return KQ8_ERR_INVALID_ARG;
    if (nq % nkv != 0 || nq / nkv > MAX_G || B > 65535 || nkv > 65535) return KQ8_ERR_UNSUPPORTED;
    if (status && (uintptr_t)status % 4) return KQ8_ERR_INVALID_ARG;
    if (B == 0 || max_len == 0 || total == 0) return KQ8_OK;
    if (!out || !q || !k || !v || !cu_seqlens) return KQ8_ERR_INVALID_ARG;
    const size_t st[6] = {q_token_stride, q_head_stride, k_token_stride,
                          k_head_stride,  v_token_stride, v_head_stride};
    for (size_t x : st)
        if (x % 8 || x > MAX_STRIDE) return KQ8_ERR_INVALID_ARG;
    if ((uintptr_t)out % 16 || (uintptr_t)q % 16 || (uintptr_t)k % 16 || (uintptr_t)v % 16)
        return KQ8_ERR_INVALID_ARG;
    // the inputs are read while other rows are written
    const size_t out_bytes = rows_bytes(total, (size_t)nq * HD, nq, HD, 2);
    if (stretches_meet(out, out_bytes, q, rows_bytes(total, st[0], nq, st[1], 2)) ||
        stretches_meet(out, out_bytes, k, rows_bytes(total, st[2], nkv, st[3], 2)) ||
        stretches_meet(out, out_bytes, v, rows_bytes(total, st[4], nkv, st[5], 2)))
        return KQ8_ERR_INVALID_ARG;
    const bool bf16 = dtype == KQ8_BF16;
    const int G = nq / nkv, TQ = PR_ROWS / G;
    PromptParams p;
    std::memset(&p, 0, sizeof(p));
    int rc = row_map(&p.qmap, bf16, q, total, nq, st[0], st[1], (uint32_t)G, (uint32_t)TQ);
    if (!rc) rc = row_map(&p.kmap, bf16, k, total, nkv, st[2], st[3], 1u, PR_BLK);
    if (!rc) rc = row_map(&p.vmap, bf16, v, total, nkv, st[4], st[5], 1u, PR_BLK);
    if (rc) return rc;
    p.out = out;
    p.cu = cu_seqlens;
    p.total = total;
    p.max_len = max_len < total ? max_len : total;
    p.nq = nq;
    p.G = G;
    p.scale = scale;
    p.status = status;
    const dim3 grid((unsigned)((p.max_len + 2 * TQ - 1) / (2 * TQ)), (unsigned)nkv, (unsigned)B);
    return bf16 ? launch_prompt<true>(p, grid, (cudaStream_t)stream)
                : launch_prompt<false>(p, grid, (cudaStream_t)stream);
}
