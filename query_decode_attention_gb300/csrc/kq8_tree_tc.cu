// kq8_tree_tc.cu -- draft-tree attention for more rows (nodes x query heads of a KV
// head) than the 16- and 32-row kernel's matrix instructions carry well, on the
// 5th-generation tensor cores.
//
// Each row is computed as in kq8_tree.cu, up to 128 rows to a tile (MMA M, TMEM lanes):
//   S [128 rows x 128 tokens] = Q K^T      O [128 rows x 128 dims] += P V.
// Q's rows are the method's codes times their block scales, as fp16 with a power of two
// per row that puts the row's largest near 2^13.  Outputs of 24 and 11 bits take K's and
// V's codes as they are (exact in fp16), the tokens' scales in fp32 beside the softmax,
// and Q and the weights p * vstep as fp16 hi and lo parts (22 bits), each an MMA of its
// own.  bf16 outputs, whose own rounding is 2^-9, take Q and P at 11 bits, V already
// multiplied by its token's step (relative to a power of two per 32 tokens), 11 bits too,
// and with two tiles K as well (KCODES): each multiplier in an operand spares the softmax
// a load and an operation per score.
//
// What bounds it.  Per 128-token step shared memory carries the raw bytes in and out of
// the ring (66 KB), the widened operands in (64 KB) and, per tile, Q and K (64 KB) and V
// (32 KB) to the MMAs: 226 KB for one tile, 322 KB for two or for hi and lo, 1770 and
// 2520 cycles at 128 bytes; the MMAs themselves take 1024 and 2048 (64 each), HBM 1440
// for the step's 33 KB.  Measured, 16 x 16384 tokens, 8 KV heads (83 us of HBM): 128
// rows bf16 234 us, 256 rows 340, 128 rows fp32 339: 4100, 6000 and 6000 cycles a step.
// The schedulers issue in half of the cycles; what is left is the latency of the chain
// widen K -> S -> widen K and of the roles' own code.  Tried at 128 rows and dropped, as
// they loosen the chain and gain nothing: steps of 64 tokens (390 against 296 us), K's and
// V's raw bytes in rings of their own (226 against 221), second places of both K and V
// (275 to 291).  With few rows the mma.sync kernel moves less: see tree_plan.
//
// Sums.  The tensor core adds products to its fp32 accumulator by cutting off, so a long
// chain of steps drifts: 1.3e-5 of the output (2-norm) after 47 steps of a stream, where
// plain fp32 sums are off by 6e-6.  fp32 and fp16 outputs therefore take O out of the
// accumulator every TC_FLUSH steps and add it to a sum in memory (L2), rounded to nearest:
// 5.8e-6, for a tenth of the time (128 rows 326 -> 360 us when it came in).  For bf16 outputs the drift
// is a hundredth of their own rounding.
//
// One persistent CTA per SM takes an equal share of all steps: the lists (row tile, KV
// head, sequence) lie one behind the other and are cut where a share ends, so ragged
// lengths leave no SM without work.  A list inside one share goes straight to the
// output, the pieces of a cut one to a merge kernel.  Two streams of steps keep the
// tensor core and the softmax busy at once: with two tiles (T = 2) each tile is a
// stream; with one, the even steps are one stream and the odd steps the other, each
// with its own O, reference and sum, joined at a list's end (fp32, 128 rows: 359 us with
// one stream, 334 with two).  TMEM holds O 2 x 128 columns and S 2 x 128, the weights
// over the scores.  Roles, which meet on mbarriers:
//   warps 0-3, 4-7  softmax of stream 0, 1, one thread per row (TMEM lane), as in
//                   kq8_prompt.cu; the reference m refers to weights (score + log2 of
//                   the V step), so that they fit fp16 whatever the V steps are;
//   warps 8-11      widen one 32-token sub-tile of K each of a step to fp16;
//   warps 12-15     the same of V;
//   warp 16         one lane issues S, the streams in turn;
//   warps 17, 18    one lane each issues PV of a tile (of one tile: 17, the streams in
//                   turn);
//   warp 19         copies raw sub-tiles (codes and scales) into a ring.
// A list's start is on every share's path: its Q is quantised 8 lanes to a row with the
// loads of 8 rows in flight (a row at a time by a whole warp: 268 us at 128 rows and 402
// at 256 instead of 221 and 342).
// Order of tokens.  Row r of a 32-token sub-tile's operands holds K position rho(r)
// (bits 1 and 2 swapped), token krow(rho(r)): with it the copies from the raw tile
// (contiguous 512 bytes an instruction) to the swizzled operand rows are free of bank
// conflicts on both sides.
#include "kq8_internal.h"
#include "kq8_quant.cuh"
#include "kq8_tc.cuh"
#include "kq8_tree.cuh"

namespace kq8 {
namespace {

constexpr int TC_STEP = 128;                     // tokens per step
constexpr int TC_THREADS = 20 * 32;
constexpr int TC_W_WIDEN = 8, TC_W_S = 16, TC_W_PV = 17, TC_W_LOAD = 19;
// registers per thread, 96 at launch: 2 * 136 + 2 * 64 + 80 = 5 * 96
constexpr int TC_REGS_SOFTMAX = 136, TC_REGS_WIDEN = 64, TC_REGS_REST = 80;
constexpr uint32_t TC_PANEL = TC_STEP * 128;     // 128 rows x 64 fp16
constexpr uint32_t TC_OP = 2 * TC_PANEL;         // an operand: 128 rows x 128 fp16
constexpr float TC_M_INIT = -1e30f;              // reference of a row that saw nothing
// hi and lo parts: O leaves the accumulator after so many steps of a stream
constexpr int TC_FLUSH = 16;
constexpr float TC_TOP = 15.0f, TC_AIM = 7.0f;   // weights stay below 2^15, are set to 2^7

template <int T, bool HILO>
struct TcShape {
    static_assert(T == 1 || !HILO, "hi and lo parts of one tile");
    static constexpr int NR = 128 * T;                 // rows of a list
    // Rings, as far as shared memory goes.  A parity wait is only sound for a waiter
    // that waits for every phase of a barrier, in order, or knows the phase before to be
    // over (the softmax, which waits for PV at a list's end only: S of that step had
    // waited for the step before's).  So the raw ring is a multiple of four long (a place
    // has the same two consumers, sub-tile w's K and V warp).
    // One tile and one part leave room for a second place of K or of V; V's it is:
    // 128 rows of 16 x 16384 tokens took 268 us so, 292 with K's.  Raw places given up
    // for either cost more than it gains.
    static constexpr int RAWN = 8, KB = 1, VB = T == 1 && !HILO ? 2 : 1;
    static constexpr uint32_t Q = 0, K = (T + (HILO ? 1 : 0)) * TC_OP, V = K + KB * TC_OP,
                              RAW = V + VB * TC_OP,
                              SC = RAW + RAWN * STAGE_BYTES,  // [4][3][128] floats
                              // [4][4]: something is missing or not finite, a bound of log2
                              // of the V steps, K's factor
                              META = SC + 4 * 3 * 512,
                              RF = META + 4 * 4 * 16,         // [T][128] row factors
                              EX = RF + T * 512,              // [2][128] (m, sum)
                              MISC = EX + 2048,               // TMEM, abort, flags, share
                              BAR = MISC + 128, SMEM = BAR + 512 + 1024;
    // barriers
    static constexpr int B_RAWF = 0, B_RAWE = B_RAWF + RAWN, B_KF = B_RAWE + RAWN,
                         B_KE = B_KF + KB, B_VF = B_KE + KB, B_VE = B_VF + VB, B_SCF = B_VE + VB,
                         B_SF = B_SCF + 4,   // [stream]
                         B_P = B_SF + 2,     // [stream][half]
                         B_PV = B_P + 4,     // [stream]
                         B_QF = B_PV + 2, B_XF = B_QF + 1, B_XE = B_XF + 1,
                         B_FINAL = B_XE + 1, B_COUNT = B_FINAL + 3;
    static_assert(B_COUNT * 8 <= 512 && SMEM <= 232448 && RAWN % 4 == 0, "shape");
};

__device__ __forceinline__ int tc_rho(int r) { return (r & ~6) | ((r & 2) << 1) | ((r & 4) >> 1); }

// 8 int8 codes -> 8 fp16: exactly, or times f (an fp16 pair of equals), or times f + fl
// with one rounding.  The last is K's: a token's factor of 11 bits would move all its
// scores by 2^-12 of themselves, which the rounding of 128 products does not.
template <bool EXACT, bool LOW = false>
__device__ __forceinline__ uint4 widen8(uint32_t a, uint32_t b, uint32_t f, uint32_t fl = 0u) {
    const uint32_t u = a ^ 0x80808080u, v = b ^ 0x80808080u;
    auto half = [&](uint32_t w, uint32_t sel) {
        const uint32_t x = hsub2(__byte_perm(w, 0x64646464u, sel), 0x64806480u);
        if (EXACT) return x;
        uint32_t r;
        if (LOW) {
            asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(fl));
            asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(r) : "r"(x), "r"(f));
        } else {
            asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(f));
        }
        return r;
    };
    return make_uint4(half(u, 0x4140), half(u, 0x4342), half(v, 0x4140), half(v, 0x4342));
}
__device__ __forceinline__ uint32_t make_half2_bits(float x) { return f2_to_h2(x, x); }
__device__ __forceinline__ void tc_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A call's lists and the CTAs' shares of their steps.  Sequence b has lists of
// seq_steps(b) steps, one for each KV head and row tile that holds a node; global
// step numbers run over row tiles, then heads, then sequences.
struct TcSeq {
    int n, base, nb, q0, steps, row_tiles;
    bool bad;
};
__device__ __forceinline__ TcSeq tc_seq(const TreeParams& P, int b, int NR) {
    TcSeq s;
    s.n = __ldg(P.seq_lens + b);
    s.q0 = __ldg(P.q_off + b);
    s.nb = __ldg(P.q_off + b + 1) - s.q0;
    s.bad = s.n < 0 || s.n > P.max_seq_len || s.nb < 0 || s.nb > s.n || s.nb > P.max_q_len ||
            s.q0 < 0 || (int64_t)s.q0 + s.nb > P.total_q;
    s.base = s.n - s.nb;
    s.steps = s.bad || s.nb == 0 ? 0 : (s.n + TC_STEP - 1) / TC_STEP;
    s.row_tiles = s.steps ? (s.nb * P.G + NR - 1) / NR : 0;
    return s;
}
// Where a CTA's share begins (in steps from the start of sequence b) and how long
// it is.  One warp, all lanes; every CTA reads all lengths.
struct TcShare {
    int64_t begin, end, total;  // global steps of the share, of all lists
    int64_t at;                 // the share's first step, counted from sequence b's first
    int b;
};
__device__ __forceinline__ int64_t tc_bound(int64_t total, int c, int ctas) {
    return total / ctas * c + total % ctas * c / ctas;
}
__device__ __forceinline__ TcShare tc_share(const TreeParams& P, int NR, int c, int ctas) {
    const int lane = threadIdx.x & 31, nkv = P.cache.num_kv_heads;
    auto seq_work = [&](int b) -> int64_t {
        if (b >= P.b0 + P.seqs) return 0;
        const TcSeq s = tc_seq(P, b, NR);
        return (int64_t)s.steps * s.row_tiles * nkv;
    };
    TcShare r;
    int64_t sum = 0;
    for (int b = P.b0 + lane; b < P.b0 + P.seqs; b += 32) sum += seq_work(b);
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    r.total = sum;
    r.begin = tc_bound(sum, c, ctas);
    r.end = tc_bound(sum, c + 1, ctas);
    r.b = P.b0;
    r.at = 0;
    int64_t before = 0;  // steps of the sequences before this round's
    for (int b0 = P.b0; b0 < P.b0 + P.seqs && r.begin < r.end; b0 += 32) {
        const int64_t w = seq_work(b0 + lane);
        int64_t upto = w;  // inclusive
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        const unsigned past = __ballot_sync(0xffffffffu, before + upto > r.begin);
        if (past) {
            const int l = __ffs(past) - 1;
            const int64_t first = __shfl_sync(0xffffffffu, before + upto - w, l);
            r.b = b0 + l;
            r.at = r.begin - first;
            break;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    return r;
}

// The pieces of a share, one list at a time; every role walks the same ones.
struct TcItem {
    TcSeq s;
    int b, h, rt;
    int step0, steps;  // this piece's steps of the list's s.steps
    __device__ bool whole() const { return steps == s.steps; }
};
struct TcWalk {
    int64_t left, at;
    int b, last_b;
    __device__ TcWalk(const TreeParams& P, const TcShare& sh)
        : left(sh.end - sh.begin), at(sh.at), b(sh.b), last_b(P.b0 + P.seqs) {}
    __device__ bool next(const TreeParams& P, int NR, TcItem& it) {
        if (left <= 0) return false;
        for (;;) {
            if (b >= last_b) return false;  // (does not happen: left counts real steps)
            it.s = tc_seq(P, b, NR);
            const int64_t work = (int64_t)it.s.steps * it.s.row_tiles * P.cache.num_kv_heads;
            if (at < work) break;
            at -= work;
            b++;
        }
        const int list = (int)(at / it.s.steps);
        it.b = b;
        it.rt = list % it.s.row_tiles;
        it.h = list / it.s.row_tiles;
        it.step0 = (int)(at % it.s.steps);
        it.steps = (int)min((int64_t)(it.s.steps - it.step0), left);
        left -= it.steps;
        at += it.steps;
        return true;
    }
};

template <int T, bool HILO>
__global__ void __launch_bounds__(TC_THREADS, 1)
    kq8_tree_tc_kernel(const __grid_constant__ TreeParams P) {
    using Sh = TcShape<T, HILO>;
    constexpr int NR = Sh::NR, RAWN = Sh::RAWN, KB = Sh::KB, VB = Sh::VB;
    // K's operand is its codes, with the tokens' multipliers beside the softmax, or their
    // product.  With one tile a step waits for the widening, with two for the softmax
    // (128 rows 231 and 256 us, 256 rows 387 and 347).
    constexpr bool KCODES = T == 1;
    constexpr bool SPLIT = T == 1;  // the streams are the even and the odd steps
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nkv = P.cache.num_kv_heads, kv_bs = P.cache.kv_bs, subs = kv_bs / TILE;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Sh::BAR);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + Sh::MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + Sh::MISC + 4);
    volatile int* sub_ok = reinterpret_cast<volatile int*>(sm + Sh::MISC + 16);  // [raw place]
    if (warp == 0) {
        __syncwarp();
        tc::tmem_alloc(tslot, 512);
    }
    if (tid == 0) {
        for (int i = 0; i < Sh::B_COUNT; i++) {
            uint32_t cnt = 1;
            if (i >= Sh::B_RAWE && i < Sh::B_KF) cnt = 2;
            if (i >= Sh::B_KF && i < Sh::B_KE) cnt = 4;
            if (i >= Sh::B_VF && i < Sh::B_VE) cnt = 4;
            if (i >= Sh::B_VE && i < Sh::B_SCF) cnt = T;  // a PV thread per tile
            if (i >= Sh::B_SCF && i < Sh::B_SF) cnt = 4;
            if (i >= Sh::B_P && i < Sh::B_PV) cnt = 4;
            if (i >= Sh::B_QF && i < Sh::B_FINAL) cnt = 8;
            mbar_init(bars + i, cnt);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    // nothing is read or written before the kernel before this one has completed
    griddep_wait();
    griddep_launch_dependents();
    TcShare* share_sm = reinterpret_cast<TcShare*>(sm + Sh::MISC + 64);
    if (warp == 1) {
        const TcShare sh = tc_share(P, NR, blockIdx.x, gridDim.x);
        if (lane == 0) *share_sm = sh;
    }
    if (blockIdx.x == 0 && warp >= 2)  // bad sequences are reported once
        for (int b = P.b0 + tid - 64; b < P.b0 + P.seqs; b += TC_THREADS - 64)
            if (tc_seq(P, b, NR).bad) atomicOr(P.status, KQ8_STATUS_BAD_SEQLEN);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tbase = *tslot;
    TcWalk walk(P, *share_sm);
    TcItem it;
    // A wait that runs out is recorded and makes every later wait that does not
    // succeed at once give up.
    auto wait = [&](int i, uint32_t parity) -> bool {
        if (mbar_try_wait(bars + i, parity)) return true;
        const long long t0 = clock64();
        while (!mbar_try_wait(bars + i, parity)) {
            if (*abort_flag) return false;
            if (clock64() - t0 > (1ll << 28)) {
                *abort_flag = 1;
                atomicOr(P.status, KQ8_STATUS_TIMEOUT);
                atomicOr(P.status + 1, 1u);  // the merge leaves every split row as it was
                return false;
            }
        }
        return true;
    };
    auto all = [](bool x) { return __all_sync(0xffffffffu, x) != 0; };
    float* sc = reinterpret_cast<float*>(sm + Sh::SC);
    float4* meta = reinterpret_cast<float4*>(sm + Sh::META);
    float* rf_sm = reinterpret_cast<float*>(sm + Sh::RF);
    // TMEM columns: O, the scores and, over them, the weights (of 16 tokens; lo 16 columns
    // on, so that a chunk of 32 tokens stays within its scores)
    auto col_o = [&](int t) { return tbase + 128 * t; };
    auto col_s = [&](int t) { return tbase + 256 + 128 * t; };
    auto off_p = [](int kk) { return HILO ? 32 * (kk >> 1) + 8 * (kk & 1) : 8 * kk; };

    if (warp >= TC_W_S) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(TC_REGS_REST));
        if (warp == TC_W_LOAD) {
            // ---- raw sub-tiles; a step always has four (past the end: empty).  Lanes
            // 4 i .. 4 i + 3 issue the copies of the step's sub-tile i: K, V and the two
            // ranges of maxima
            const uint64_t pol = P.row_tiles > 1 ? l2_evict_last_policy() : l2_evict_first_policy();
            const int i = (lane >> 2) & 3, piece = lane & 3;
            uint32_t ri = 0;  // running sub-tile
            bool ok = true;
            while (ok && walk.next(P, NR, it)) {
                const int tile0 = 4 * it.step0;
                const int tiles = min(4 * it.steps, (it.s.n + TILE - 1) / TILE - tile0);
                auto window = [&](int w) -> int32_t {  // page ids, one per lane
                    const int t = 32 * w + lane;
                    if (t >= tiles) return -1;
                    const int32_t pg =
                        P.page_table[(size_t)it.b * P.max_pages + (tile0 + t) / subs];
                    if (pg >= 0 && pg < P.cache.num_pages) return pg;
                    atomicOr(P.status, KQ8_STATUS_BAD_PAGE);
                    return -1;
                };
                int32_t cur = window(0), nxt = window(1);
                for (int t = 0; t < 4 * it.steps; t += 4, ri += 4) {
                    const int s = (ri + i) % RAWN;
                    if (ri >= (uint32_t)RAWN) {
                        ok = __all_sync(0xffffffffu, wait(Sh::B_RAWE + s, (ri / RAWN - 1) & 1));
                        if (!ok) break;
                    }
                    if ((t & 31) == 0 && t > 0) {
                        cur = nxt;
                        nxt = window((t >> 5) + 1);
                    }
                    const int32_t pg = __shfl_sync(0xffffffffu, cur, (t & 31) + i);
                    uint64_t* bar = bars + Sh::B_RAWF + s;
                    if (lane < 16 && piece == 0) {
                        sub_ok[s] = pg >= 0;
                        mbar_arrive_expect_tx(bar, pg >= 0 ? STAGE_BYTES : 0);
                    }
                    __syncwarp();
                    if (lane < 16 && pg >= 0) {
                        const int sub = (tile0 + t + i) % subs;
                        const size_t kvo = kv_sub_off(pg, it.h, nkv, kv_bs, sub);
                        const size_t so = scale_sub_off(pg, it.h, nkv, kv_bs, sub);
                        const void* src = piece == 0   ? (const void*)(P.cache.k + kvo)
                                          : piece == 1 ? (const void*)(P.cache.v + kvo)
                                          : piece == 2 ? (const void*)(P.cache.kscale + so)
                                                       : (const void*)(P.cache.vscale + so);
                        const uint32_t at = piece == 0   ? 0
                                            : piece == 1 ? SUB_K_BYTES
                                            : piece == 2 ? SUB_K_BYTES + SUB_V_BYTES
                                                         : SUB_K_BYTES + SUB_V_BYTES + SUB_S_BYTES;
                        bulk_g2s(sm + Sh::RAW + s * STAGE_BYTES + at, src,
                                 piece < 2 ? SUB_K_BYTES : SUB_S_BYTES, bar, pol);
                    }
                    __syncwarp();
                }
            }
            // every copy has landed before shared memory is given up (bounded)
            for (uint32_t k = ri > (uint32_t)RAWN ? ri - RAWN : 0; k < ri; k++)
                mbar_wait_bounded(bars + Sh::B_RAWF + k % RAWN, (k / RAWN) & 1);
        } else if (warp == TC_W_S && lane == 0) {
            // ---- S.  Operand rows are 128 bytes, swizzled; a K-major step of 16 elements
            // is 32 bytes along the row.
            const uint64_t dq = tc::sdesc_sw128(smem_u32(sm + Sh::Q), 16, 1024);
            const uint64_t dk = tc::sdesc_sw128(smem_u32(sm + Sh::K), 16, 1024);
            constexpr uint32_t IDS = tc::IDesc<128, TC_STEP, false>::value;
            uint32_t g = 0, qn = 0;    // steps, lists so far
            uint32_t n[2] = {0u, 0u};  // products of each stream so far
            bool ok = true;
            while (ok && walk.next(P, NR, it)) {
                ok = wait(Sh::B_QF, qn++ & 1);
                for (int j = 0; ok && j < it.steps; j++, g++) {
                    const int place = g % KB;
                    if (!(ok = wait(Sh::B_KF + place, (g / KB) & 1))) break;
                    const uint64_t k = dk + (uint64_t)(place * (TC_OP >> 4));
                    for (int i = 0; ok && i < T; i++) {
                        const int t = SPLIT ? (int)(g & 1) : i;
                        // the place is free when PV has read the weights over the scores
                        if (n[t] >= 1 && !(ok = wait(Sh::B_PV + t, (n[t] - 1) & 1))) break;
                        tc::fence_after_sync();
#pragma unroll
                        for (int part = 0; part < (HILO ? 2 : 1); part++) {
                            const uint64_t a = dq + (uint64_t)((i + part) * (TC_OP >> 4));
#pragma unroll
                            for (int kk = 0; kk < HD / 16; kk++) {
                                const uint64_t o = (kk >> 2) * (TC_PANEL >> 4) + (kk & 3) * 2;
                                tc::mma_f16(col_s(t), a + o, k + o, IDS, kk > 0 || part > 0);
                            }
                        }
                        tc::mma_commit(bars + Sh::B_SF + t);
                        n[t]++;
                    }
                    if (ok) tc::mma_commit(bars + Sh::B_KE + place);
                }
            }
            // every commit has arrived before the CTA may end (bounded)
            tc::mma_commit(bars + Sh::B_FINAL);
            mbar_wait_bounded(bars + Sh::B_FINAL, 0);
            for (uint32_t k = g > (uint32_t)KB ? g - KB : 0; ok && k < g; k++)
                mbar_wait_bounded(bars + Sh::B_KE + k % KB, (k / KB) & 1);
        } else if (warp >= TC_W_PV && warp < TC_W_PV + T && lane == 0) {
            // ---- PV, of a tile or of both streams in turn.  V's step of 16 tokens is two
            // groups of eight rows.
            const int tile = warp - TC_W_PV;
            const uint64_t dv = tc::sdesc_sw128(smem_u32(sm + Sh::V), TC_PANEL, 1024);
            constexpr uint32_t IDO = tc::IDesc<128, HD, false>::value | tc::IDESC_B_MN;
            uint32_t g = 0;            // steps so far
            bool ok = true;
            while (ok && walk.next(P, NR, it)) {
                for (int j = 0; ok && j < it.steps; j++, g++) {
                    const int place = g % VB, t = SPLIT ? (int)(g & 1) : tile;
                    const uint32_t m = SPLIT ? g >> 1 : g;  // of the stream
                    const bool first = HILO ? (j >> 1) % TC_FLUSH == 0 : j < (SPLIT ? 2 : 1);
                    const uint64_t v = dv + (uint64_t)(place * (TC_OP >> 4));
                    ok = wait(Sh::B_VF + place, (g / VB) & 1);
#pragma unroll
                    for (int half = 0; half < 2; half++) {
                        if (!(ok = ok && wait(Sh::B_P + 2 * t + half, m & 1))) break;
                        tc::fence_after_sync();
#pragma unroll
                        for (int kk = 4 * half; kk < 4 * half + 4; kk++) {
                            const uint64_t b = v + (uint64_t)(kk * (2048 >> 4));
                            const uint32_t p = col_s(t) + off_p(kk);
                            tc::mma_f16_ta(col_o(t), p, b, IDO, !first || kk > 0);
                            if (HILO) tc::mma_f16_ta(col_o(t), p + 16, b, IDO, true);
                        }
                    }
                    if (!ok) break;
                    tc::mma_commit(bars + Sh::B_PV + t);
                    tc::mma_commit(bars + Sh::B_VE + place);
                }
            }
            tc::mma_commit(bars + Sh::B_FINAL + 1 + tile);
            mbar_wait_bounded(bars + Sh::B_FINAL + 1 + tile, 0);
            for (uint32_t k = g > (uint32_t)VB ? g - VB : 0; ok && k < g; k++)
                mbar_wait_bounded(bars + Sh::B_VE + k % VB, (k / VB) & 1);
        }
    } else if (warp >= TC_W_WIDEN) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(TC_REGS_WIDEN));
        const int w = (warp - TC_W_WIDEN) & 3;  // sub-tile of a step
        const bool is_v = warp >= TC_W_WIDEN + 4;
        const float kmul = inv127() * P.scale * TR_LOG2E;
        // a power of two above x (finite, >= 0)
        auto above = [](float x) { return min(max((int)(__float_as_uint(x) >> 23) - 126, -90), 100); };
        uint32_t g = 0;
        bool ok = true;
        while (ok && walk.next(P, NR, it)) {
            for (int j = 0; j < it.steps; j++, g++) {
                const uint32_t ri = 4 * g + w;
                const int s = ri % RAWN, place = g % (is_v ? VB : KB);
                if (!(ok = all(wait(Sh::B_RAWF + s, (ri / RAWN) & 1)))) break;
                const uint8_t* st = sm + Sh::RAW + s * STAGE_BYTES;
                // lane = operand row: its token's K multiplier or V step
                const int tok = krow(tc_rho(lane));
                const float* rs = reinterpret_cast<const float*>(st + SUB_K_BYTES + SUB_V_BYTES);
                const bool have = sub_ok[s] != 0;
                const bool live = have && (4 * (it.step0 + j) + w) * TILE + tok < it.s.n;
                // a token past the end or on a missing page counts for nothing
                const float km = live ? __fmul_rn(rs[tok], kmul) : 0.0f;
                const float vstep = live ? __fmul_rn(rs[32 + tok], inv127()) : 0.0f;
                const uint32_t vb = __float_as_uint(fabsf(vstep)) < 0x7F800000u
                                        ? __float_as_uint(fabsf(vstep)) : 0u;
                const int ve = above(__uint_as_float(__reduce_max_sync(0xffffffffu, vb)));
                if (!is_v) {
                    const uint32_t kb = __float_as_uint(fabsf(km)) < 0x7F800000u
                                            ? __float_as_uint(fabsf(km)) : 0u;
                    const int ke = above(__uint_as_float(__reduce_max_sync(0xffffffffu, kb)));
                    const bool odd = !have || __any_sync(0xffffffffu, !(fabsf(vstep) < INFINITY));
                    if (g >= (uint32_t)KB && !(ok = all(wait(Sh::B_KE + place, (g / KB - 1) & 1)))) break;
                    // (The place of the step's scales was last read for step g - 4.  Before
                    // S(g - KB) PV had read the weights of step g - KB - 2 and all before it.)
                    static_assert(KB <= 2, "scales");
                    float* d = sc + (g & 3) * 384 + 32 * w + lane;
                    d[0] = km;
                    d[128] = vstep;
                    float lv;  // log2 of the V step, from below
                    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lv) : "f"(vstep));
                    lv = lv < 128.0f ? fmaxf(lv, -90.0f) : INFINITY;  // not finite: the row is lost
                    d[256] = have ? lv : -INFINITY;                   // a missing page's: masked
                    if (lane == 0)
                        meta[(g & 3) * 4 + w] = make_float4(odd ? 1.0f : 0.0f, (float)ve,
                                                            KCODES ? 1.0f : pow2i(ke), 0.0f);
                    // K: lane = (position pair, 16-byte half); its 16 codes are chunks c, c + 1
                    // of the row's panel
                    const float fk = km * pow2i(-ke);
                    const uint32_t f = make_half2_bits(fk);
                    const uint32_t fl = make_half2_bits(fk - h2_to_f2(f).x);
                    const int rowa = 32 * w + tc_rho(lane >> 1), x7 = rowa & 7;
                    const uint32_t fa = __shfl_sync(0xffffffffu, f, rowa & 31);
                    const uint32_t fb = __shfl_sync(0xffffffffu, f, (rowa + 16) & 31);
                    const uint32_t fla = __shfl_sync(0xffffffffu, fl, rowa & 31);
                    const uint32_t flb = __shfl_sync(0xffffffffu, fl, (rowa + 16) & 31);
                    uint4 xa = *reinterpret_cast<const uint4*>(st + 16 * lane);
                    uint4 xb = *reinterpret_cast<const uint4*>(st + 512 + 16 * lane);
#pragma unroll 1
                    for (int blk = 0; blk < 4; blk++) {
                        const uint4 ya = xa, yb = xb;
                        if (blk < 3) {
                            xa = *reinterpret_cast<const uint4*>(st + 1024 * (blk + 1) + 16 * lane);
                            xb = *reinterpret_cast<const uint4*>(st + 1024 * (blk + 1) + 512 + 16 * lane);
                        }
                        const int c = (blk & 1) * 4 + (lane & 1) * 2;
                        uint8_t* o = sm + Sh::K + place * TC_OP + (blk >> 1) * TC_PANEL + rowa * 128;
                        const int c0 = (c ^ x7) << 4, c1 = ((c + 1) ^ x7) << 4;
                        *reinterpret_cast<uint4*>(o + c0) = widen8<KCODES, true>(ya.x, ya.y, fa, fla);
                        *reinterpret_cast<uint4*>(o + c1) = widen8<KCODES, true>(ya.z, ya.w, fa, fla);
                        *reinterpret_cast<uint4*>(o + 2048 + c0) = widen8<KCODES, true>(yb.x, yb.y, fb, flb);
                        *reinterpret_cast<uint4*>(o + 2048 + c1) = widen8<KCODES, true>(yb.z, yb.w, fb, flb);
                    }
                } else {
                    if (g >= (uint32_t)VB && !(ok = all(wait(Sh::B_VE + place, (g / VB - 1) & 1)))) break;
                    // V: tokens t and t + 4 (neighbouring positions), one panel each; a step that
                    // is not finite counts as 0 here (the softmax sees to the rows that see it)
                    const uint32_t f =
                        make_half2_bits(fabsf(vstep) < INFINITY ? vstep * pow2i(-ve) : 0.0f);
                    const int a = (lane >> 2) & 1, q = lane & 3, p = a ^ ((lane >> 3) & 1);
                    const int u = (lane >> 4) + 4 * a;  // tokens 8 i + u and + 2
                    const uint8_t* src = st + SUB_K_BYTES + u * HD + 64 * p + 16 * q;
                    uint8_t* dst = sm + Sh::V + place * TC_OP + p * TC_PANEL + 32 * w * 128;
                    uint4 xa = *reinterpret_cast<const uint4*>(src);
                    uint4 xb = *reinterpret_cast<const uint4*>(src + 2 * HD);
#pragma unroll 1
                    for (int i = 0; i < 4; i++) {
                        const uint4 ya = xa, yb = xb;
                        if (i < 3) {
                            xa = *reinterpret_cast<const uint4*>(src + (8 * i + 8) * HD);
                            xb = *reinterpret_cast<const uint4*>(src + (8 * i + 10) * HD);
                        }
                        const int ra = tc_rho(kpos(8 * i + u)), rb = tc_rho(kpos(8 * i + u + 2));
                        const uint32_t fa = __shfl_sync(0xffffffffu, f, ra);
                        const uint32_t fb = __shfl_sync(0xffffffffu, f, rb);
                        uint8_t *oa = dst + ra * 128, *ob = dst + rb * 128;
                        *reinterpret_cast<uint4*>(oa + (((2 * q) ^ (ra & 7)) << 4)) =
                            widen8<HILO>(ya.x, ya.y, fa);
                        *reinterpret_cast<uint4*>(oa + (((2 * q + 1) ^ (ra & 7)) << 4)) =
                            widen8<HILO>(ya.z, ya.w, fa);
                        *reinterpret_cast<uint4*>(ob + (((2 * q) ^ (rb & 7)) << 4)) =
                            widen8<HILO>(yb.x, yb.y, fb);
                        *reinterpret_cast<uint4*>(ob + (((2 * q + 1) ^ (rb & 7)) << 4)) =
                            widen8<HILO>(yb.z, yb.w, fb);
                    }
                }
                tc::fence_smem_to_async();
                __syncwarp();
                if (lane == 0) {
                    tc_arrive(bars + Sh::B_RAWE + s);
                    if (!is_v) tc_arrive(bars + Sh::B_SCF + (g & 3));
                    tc_arrive(bars + (is_v ? Sh::B_VF : Sh::B_KF) + place);
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(TC_REGS_SOFTMAX));
        const int t = warp >> 2, w4 = warp & 3;  // stream
        const int row = w4 * 32 + lane;          // of its tile
        const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
        const uint32_t tO = col_o(t) + lanes, tS = col_s(t) + lanes;
        float2* ex = reinterpret_cast<float2*>(sm + Sh::EX);
        float* spill = HILO ? P.spill + ((size_t)blockIdx.x * 2 + t) * HD * 128 + row : nullptr;
        uint32_t g = 0, n = 0, xn = 0;  // steps, this stream's steps, lists so far
        bool ok = true;
        for (int piece = 0; ok && walk.next(P, NR, it); piece++) {
            const int tile = T == 2 ? t : 0;
            const int r0 = it.rt * NR + 128 * tile;        // first row of the tile
            const int rows = it.s.nb * P.G - r0;           // of the tile (may be <= 0 or > 128)
            // ---- Q (article 9-2 §2 seg. 1): codes times block scales, scaled per row.
            // Stream t of a split tile prepares half of it.  (With one tile the streams
            // have met since their last scores, below.)
            // 8 lanes a row, 16 elements a lane, the loads of 8 rows in flight together.
            constexpr int QR = SPLIT ? 16 : 32;            // rows per warp
#pragma unroll 1
            for (int i = 0; i < QR; i += 8) {
                float4 x[2][4];
                load_type<HILO>(P.dtype, [&](auto type) {
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        const int r = (SPLIT ? 64 * t : 0) + w4 * QR + i + 4 * u + (lane >> 3);
                        const unsigned rr = (unsigned)(r0 + r), nd = rr / (unsigned)P.G;
                        const int64_t at = (int64_t)(it.s.q0 + (int)nd) * P.q_st +
                                           (int64_t)(it.h * P.G + (int)(rr - nd * P.G)) * P.q_sh +
                                           16 * (lane & 7);
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            x[u][k] = r < rows ? load_q4(P.q, decltype(type)::value, at + 4 * k)
                                               : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    }
                });
#pragma unroll
                for (int u = 0; u < 2; u++) {
                    const int r = (SPLIT ? 64 * t : 0) + w4 * QR + i + 4 * u + (lane >> 3);
                    float v[16];
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        v[4 * k] = x[u][k].x;
                        v[4 * k + 1] = x[u][k].y;
                        v[4 * k + 2] = x[u][k].z;
                        v[4 * k + 3] = x[u][k].w;
                    }
                    float m = 0.0f;
#pragma unroll
                    for (int k = 0; k < 16; k++) m = fmaxf(m, fabsf(v[k]));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                    if (m < 1e-6f) m = 1.0f;
                    const float iq = __fdiv_rn(127.0f, m);
                    const float qs = __fmul_rn(m, inv127());
                    float top = qs;
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                    // 127 * top in [2^13, 2^14) after the scale
                    const int e = min(max((int)(__float_as_uint(top) >> 23) - 127 + 7 - 13, -100), 100);
                    if ((lane & 7) == 0) rf_sm[128 * tile + r] = pow2i(e);
                    const float f = qs * pow2i(-e);
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        float y[2];
#pragma unroll
                        for (int d = 0; d < 2; d++) {
                            const float c = fminf(fmaxf(__fmul_rn(v[2 * k + d], iq), -128.0f), 127.0f);
                            y[d] = truncf(c) * f;
                        }
                        hi[k] = f2_to_h2(y[0], y[1]);
                        if (HILO) {
                            const float2 h = h2_to_f2(hi[k]);
                            lo[k] = f2_to_h2(y[0] - h.x, y[1] - h.y);
                        }
                    }
                    uint8_t* o = sm + Sh::Q + tile * TC_OP + ((lane >> 2) & 1) * TC_PANEL + r * 128;
                    const int c0 = ((2 * (lane & 3)) ^ (r & 7)) << 4, c1 = ((2 * (lane & 3) + 1) ^ (r & 7)) << 4;
                    *reinterpret_cast<uint4*>(o + c0) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(o + c1) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
                    if (HILO) {
                        *reinterpret_cast<uint4*>(o + TC_OP + c0) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        *reinterpret_cast<uint4*>(o + TC_OP + c1) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
                    }
                }
            }
            tc::fence_smem_to_async();
            __syncwarp();
            if (lane == 0) tc_arrive(bars + Sh::B_QF);
            // the row factors of both streams' halves (and, in time, O's readers below)
            if (!(ok = all(wait(Sh::B_QF, xn & 1)))) break;
            const float rf = rf_sm[128 * tile + row];
            const int node = (r0 + row) / P.G;
            float M = TC_M_INIT;
            float sum = 0.0f;
            bool first = true, spilled = false;
            float M_spill = 0.0f;  // the reference of what has been spilled
            for (int j = 0; ok && j < it.steps; j++, g++) {
                if (SPLIT && (int)(g & 1) != t) continue;
                const float* km = sc + (g & 3) * 384;
                if (!(ok = all(wait(Sh::B_SCF + (g & 3), (g >> 2) & 1)))) break;
                const int tile0 = 4 * (it.step0 + j);  // the step's first sub-tile
                const float4* mt = meta + (g & 3) * 4;
                const bool masked = (tile0 + 4) * TILE > it.s.base || mt[0].x + mt[1].x + mt[2].x + mt[3].x != 0.0f;
                auto window = [&](int w) -> uint32_t {
                    return row < rows ? node_window(P, it.s.q0, node, it.s.nb,
                                                    (tile0 + w) * TILE - it.s.base)
                                      : 0u;
                };
                // hi and lo parts: the row's windows, all loads in flight while S is made.  (Their
                // four registers cost the bf16 forms, with less work a step, more than that:
                // 128 rows 232 -> 268 us.)
                uint32_t win[4] = {0u, 0u, 0u, 0u};
                if (HILO && masked) {
#pragma unroll
                    for (int w = 0; w < 4; w++) win[w] = window(w);
                }
                if (!(ok = all(wait(Sh::B_SF + t, n & 1)))) break;
                tc::fence_after_sync();
                bool lost = false;  // the row sees a V step that is not finite
                // columns 32 w .. + 31: x * f is the score (base 2), -inf where the row does not
                // see the token; top bounds the exponents of the V steps that it sees
                auto fetch = [&](int w, float (&x)[32], float& f, float& top) {
                    tc::tmem_ld32(tS + 32 * w, x);
                    const float4 m = mt[w];
                    f = rf * m.z;
                    top = m.y;
                    if (KCODES) {
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const float4 k4 = *reinterpret_cast<const float4*>(km + 32 * w + c);
                            const float2 a =
                                __fmul2_rn(make_float2(x[c], x[c + 1]), make_float2(k4.x, k4.y));
                            const float2 b =
                                __fmul2_rn(make_float2(x[c + 2], x[c + 3]), make_float2(k4.z, k4.w));
                            x[c] = a.x;
                            x[c + 1] = a.y;
                            x[c + 2] = b.x;
                            x[c + 3] = b.y;
                        }
                    }
                    if (masked) {
                        const uint32_t on_w = !HILO ? window(w)
                                              : w < 2 ? (w == 0 ? win[0] : win[1])
                                                      : (w == 2 ? win[2] : win[3]);
                        float most = -90.0f;
#pragma unroll
                        for (int c = 0; c < 32; c++) {
                            const float l = km[256 + 32 * w + c];
                            const bool on = ((on_w >> krow(tc_rho(c))) & 1u) && l > -INFINITY;
                            lost |= on && l == INFINITY;
                            if (on && l < INFINITY) most = fmaxf(most, l);
                            x[c] = on ? x[c] : -INFINITY;
                        }
                        if (HILO) top = most + 1.0f;
                    }
                };
                float far = -INFINITY;  // a bound of the row's weights' exponents
#pragma unroll 1
                for (int w = 0; w < 4; w++) {
                    float x[32], f, top;
                    fetch(w, x, f, top);
                    float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                    for (int c = 4; c < 32; c += 8)
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            m4[i] = fmaxf(m4[i], c + 4 + i < 32 ? fmaxf(x[c + i], x[c + 4 + i]) : x[c + i]);
                    far = fmaxf(far, fmaf(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), f, top));
                }
                const bool need = far > M + TC_TOP;
                // (PV of the stream's step before is in O: S went over its weights.)
                if (HILO && j >= 2 && (j >> 1) % TC_FLUSH == 0) {
                    const float f = tr_ex2(M_spill - M);
#pragma unroll 1
                    for (int c = 0; c < HD / 32; c++) {
                        float o[32], a[32];
                        float* at = spill + 32 * c * 128;
                        if (spilled) {
#pragma unroll
                            for (int i = 0; i < 32; i++) a[i] = __ldcg(at + 128 * i);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; i++) a[i] = 0.0f;
                        }
                        tc::tmem_ld32(tO + 32 * c, o);
#pragma unroll
                        for (int i = 0; i < 32; i++) __stcg(at + 128 * i, fmaf(a[i], f, o[i]));
                    }
                    M_spill = M;
                    spilled = first = true;
                }
                if (__any_sync(0xffffffffu, need)) {
                    const float m = need ? far - TC_AIM : M;
                    const float f = tr_ex2(M - m);
                    M = m;
                    sum *= f;
                    if (!first) {
#pragma unroll 1
                        for (int c = 0; c < HD / 32; c++) {
                            float o[32];
                            tc::tmem_ld32(tO + 32 * c, o);
#pragma unroll
                            for (int i = 0; i < 32; i++) o[i] *= f;
                            tc::tmem_st32(tO + 32 * c, o);
                        }
                    }
                }
                first = false;
#pragma unroll 1
                for (int w = 0; w < 4; w++) {
                    float x[32], f, top;
                    fetch(w, x, f, top);
                    // bf16: p * 2^(the sub-tile's V exponent) is the weight itself
                    const float ve = HILO ? 0.0f : mt[w].y;
                    const float2 f2 = make_float2(f, f), o2 = make_float2(ve - M, ve - M);
                    float2 s2 = make_float2(0.0f, 0.0f);
                    float hi[16], lo[16];  // 16 columns of fp16 pairs
#pragma unroll
                    for (int i = 0; i < 16; i++) {
                        const float2 y = __ffma2_rn(make_float2(x[2 * i], x[2 * i + 1]), f2, o2);
                        const float2 p = make_float2(tr_ex2(y.x), tr_ex2(y.y));
                        s2 = __fadd2_rn(s2, p);
                        float2 wt = p;
                        if (HILO) {
                            wt = __fmul2_rn(p, *reinterpret_cast<const float2*>(km + 128 + 32 * w + 2 * i));
                            if (masked) {  // a masked token's V step may be anything
                                wt.x = p.x == 0.0f ? 0.0f : wt.x;
                                wt.y = p.y == 0.0f ? 0.0f : wt.y;
                            }
                        }
                        const uint32_t h = f2_to_h2(wt.x, wt.y);
                        hi[i] = __uint_as_float(h);
                        if (HILO) {
                            const float2 b = h2_to_f2(h);
                            lo[i] = __uint_as_float(f2_to_h2(wt.x - b.x, wt.y - b.y));
                        }
                    }
                    sum = fmaf(s2.x + s2.y, pow2i(-(int)ve), sum);
                    tc::tmem_st16(tS + off_p(2 * w), hi);
                    if (HILO) tc::tmem_st16(tS + off_p(2 * w) + 16, lo);
                    if (w & 1) {  // half of the weights, of which the product may begin
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) tc_arrive(bars + Sh::B_P + 2 * t + (w >> 1));
                    }
                }
                if (lost) sum = NAN;
                n++;
            }
            if (!ok) break;
            if (!first) {
                if (!(ok = all(wait(Sh::B_PV + t, (n - 1) & 1)))) break;
                tc::fence_after_sync();
            }
            if (HILO && spilled) {
                const float f = tr_ex2(M_spill - M);
#pragma unroll 1
                for (int c = 0; c < HD / 32; c++) {
                    float o[32], a[32];
#pragma unroll
                    for (int i = 0; i < 32; i++) a[i] = __ldcg(spill + (32 * c + i) * 128);
                    tc::tmem_ld32(tO + 32 * c, o);
#pragma unroll
                    for (int i = 0; i < 32; i++) o[i] = fmaf(a[i], f, o[i]);
                    tc::tmem_st32(tO + 32 * c, o);
                }
            }
            // ---- the list's result.  The streams of one tile meet: each then writes half
            // of the dimensions from both O's.
            float den = sum;
            float f[2] = {1.0f, 0.0f};
            if (SPLIT) {
                ex[128 * t + row] = make_float2(M, den);
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc_arrive(bars + Sh::B_XF);
                if (!(ok = all(wait(Sh::B_XF, xn & 1)))) break;
                tc::fence_after_sync();
                const float2 a = ex[row], b = ex[128 + row];
                M = fmaxf(a.x, b.x);
                f[0] = a.y == 0.0f ? 0.0f : tr_ex2(a.x - M);
                f[1] = b.y == 0.0f ? 0.0f : tr_ex2(b.x - M);
                den = a.y * f[0] + b.y * f[1];
            }
            // a share cuts at most its first and its last list
            const size_t at = (((size_t)blockIdx.x * 2 + (piece == 0 ? 0 : 1)) * NR + 128 * tile + row);
            const bool mine = row < rows;
            const float inv = it.whole() ? (den == 0.0f ? 0.0f : __fdiv_rn(1.0f, den)) : 1.0f;
            const size_t out = ((size_t)(it.s.q0 + node) * P.nq + (size_t)it.h * P.G +
                                (r0 + row) % P.G) * HD;
#pragma unroll 1
            for (int c = SPLIT ? 2 * t : 0; c < (SPLIT ? 2 * t + 2 : 4); c++) {
                float o[32];
                tc::tmem_ld32((SPLIT ? col_o(0) + lanes : tO) + 32 * c, o);
                if (SPLIT) {
                    float o1[32];
                    tc::tmem_ld32(col_o(1) + lanes + 32 * c, o1);
#pragma unroll
                    for (int i = 0; i < 32; i++)  // a stream without steps left nothing there
                        o[i] = (f[0] == 0.0f ? 0.0f : o[i] * f[0]) + (f[1] == 0.0f ? 0.0f : o1[i] * f[1]);
                } else if (den == 0.0f) {
#pragma unroll
                    for (int i = 0; i < 32; i++) o[i] = 0.0f;
                }
                if (mine) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 y = make_float4(o[i] * inv, o[i + 1] * inv, o[i + 2] * inv,
                                                     o[i + 3] * inv);
                        if (it.whole())
                            store_out4(P.out, P.dtype, out + 32 * c + i, y);
                        else
                            *reinterpret_cast<float4*>(P.part_acc + at * HD + 32 * c + i) = y;
                    }
                }
            }
            if (mine && !it.whole() && (!SPLIT || t == 0)) P.part_ms[at] = make_float2(M, den);
            tc::fence_before_sync();
            if (SPLIT) {
                // both O's and the exchange are read before either is written again
                __syncwarp();
                if (lane == 0) tc_arrive(bars + Sh::B_XE);
                if (!(ok = all(wait(Sh::B_XE, xn & 1)))) break;
            }
            xn++;
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        __syncwarp();
        tc::fence_after_sync();
        tc::tmem_dealloc(tbase, 512);
    }
}

// The lists that shares have cut:
//   m = max_c m_c, out = sum_c acc_c 2^(m_c - m) / sum_c S_c 2^(m_c - m).
// Block (c, y) merges rows 8 y .. of the list that ends inside share c but began
// before it, a warp per row.  A CTA's piece is its part 0 if it is the share's first,
// else part 1.  After a CTA has given up (some parts are missing) every row stays as
// it was; the mark goes with kq8_workspace_init, which a failed call asks for.
constexpr int TM_WARPS = 8;
__global__ void __launch_bounds__(TM_WARPS * 32)
    kq8_tree_merge_kernel(const __grid_constant__ TreeParams P, const int NR) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ctas = gridDim.x;
    __shared__ TcShare share_sm;
    if (warp == 0) {
        const TcShare sh = tc_share(P, NR, blockIdx.x, ctas);
        if (lane == 0) share_sm = sh;
    }
    __syncthreads();
    const TcShare sh = share_sm;
    TcWalk walk(P, sh);
    TcItem it;
    if (P.status[1] != 0u || !walk.next(P, NR, it)) return;
    if (it.step0 == 0 || it.step0 + it.steps < it.s.steps) return;
    const int row = blockIdx.y * TM_WARPS + warp, rr = it.rt * NR + row;
    if (row >= NR || rr >= it.s.nb * P.G) return;
    const int64_t first = sh.begin - it.step0;  // the list's first step
    int c = (int)blockIdx.x;
    float m = TC_M_INIT, den = 0.0f;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (;; c--) {
        const int64_t begin = tc_bound(sh.total, c, ctas);
        const int64_t end = tc_bound(sh.total, c + 1, ctas);
        if (begin < end) {  // a share of nothing wrote nothing
            const size_t at = ((size_t)c * 2 + (begin < first ? 1 : 0)) * NR + row;
            const float2 ms = P.part_ms[at];
            const float4 x = reinterpret_cast<const float4*>(P.part_acc + at * HD)[lane];
            const float mn = fmaxf(m, ms.x);
            const float fo = tr_ex2(m - mn), fn = tr_ex2(ms.x - mn);
            den = den * fo + ms.y * fn;
            a.x = a.x * fo + x.x * fn;
            a.y = a.y * fo + x.y * fn;
            a.z = a.z * fo + x.z * fn;
            a.w = a.w * fo + x.w * fn;
            m = mn;
        }
        if (begin <= first) break;
    }
    const float inv = den == 0.0f ? 0.0f : 1.0f, dv = den == 0.0f ? 1.0f : den;
    store_out4(P.out, P.dtype,
               ((size_t)(it.s.q0 + rr / P.G) * P.nq + (size_t)it.h * P.G + rr % P.G) * HD + 4 * lane,
               make_float4(a.x / dv * inv, a.y / dv * inv, a.z / dv * inv, a.w / dv * inv));
}

template <int T, bool HILO>
int launch_tc(const TreeParams& p, int ctas, cudaStream_t s) {
    static std::atomic<uint64_t> opted{0};
    return launch_smem(kq8_tree_tc_kernel<T, HILO>, opted, dim3((unsigned)ctas), TC_THREADS,
                       TcShape<T, HILO>::SMEM, s, p);
}

}  // namespace

int launch_tree_tc(const TreeParams& p, int tile_rows, int ctas, cudaStream_t s) {
    int rc = p.dtype != KQ8_BF16 ? launch_tc<1, true>(p, ctas, s)
             : tile_rows == 128  ? launch_tc<1, false>(p, ctas, s)
                                 : launch_tc<2, false>(p, ctas, s);
    if (rc || ctas == 1) return rc;
    return launch_pdl(kq8_tree_merge_kernel, dim3((unsigned)ctas, (unsigned)(tile_rows / TM_WARPS)),
                      TM_WARPS * 32, s, p, tile_rows);
}

}  // namespace kq8
