// Backward of the sliding-window attention with sink tokens on the tensor cores (bf16).
//
//   p_ij = 2^(c s_ij - lse_i log2 e), c = scale log2 e;  delta_i = dy_i . y_i
//   dS_ij = p_ij (dy_i . v_j - delta_i)
//   dq_i = scale sum_j dS_ij k_j, dk_j = scale sum_i dS_ij q_i, dv_j = sum_i p_ij dy_i
//
// Two persistent kernels. Both form the scores again, so that
// every output row belongs to one block and nothing is added atomically (7 products
// per tile pair instead of 5).
//   DQ   unit = a query tile of a head; steps = the sink block, then its key tiles:
//        S = Q K^T, X = dY V^T, dQ += dS K. Two warps of their own form delta one unit
//        ahead; -lse log2 e and delta, padded to whole tiles, go to the workspace.
//   DKV  unit = a key tile of a key/value head; steps = (head of the group, query
//        tile): S = K Q^T, X = V dY^T, dV += P dY, dK += dS Q (P, dS transposed: rows
//        are keys). The sinks' pairs outside the window are units of their own, whose
//        fp32 partials a last launch joins (see SinkSplit).
//
// delta = dy . y takes the forward's y as it was rounded. With few visible keys that
// error is large beside dP - delta (dq off by 0.0044 of its size at w = 2, 0.0027 at 12,
// 0.0025 at 64), and rows with few keys have the largest gradients. So DQ sweeps the steps
// of a tile twice where its first row sees fewer than 64 keys (small windows, the first
// tile of every sequence), and takes delta = sum_j p_ij dP_ij in fp32 from the first sweep
// (0.0024 at any w). The second sweep of the first tiles costs a few steps per sequence; where
// every tile takes it, with w + n_sink below 64, 8 x 16 heads x 2048 x 64, w = 32, 4 sinks takes
// 165 us with it and 134 without (at d = 128, 2 x 16 (4) x 8192, w = 16, 264 and 306: there the
// sweeps are shorter than the wait for the delta warps).
//
// P and dS are rounded to bf16, the products' operand type: at most 2^-8 of each element,
// independent from one to the next (0.0017 of dq, dk, dv). They overlay the S and X they
// come from, so the accumulators fit beside them.
// The rows work in two phases, weights (which need S) and dS (which needs X), and the
// tensor core runs one phase's products during the other: DKV issues dV(n), S(n + 1)
// once the weights of step n stand, dK(n), X(n + 1) once its dS stand; DQ has two S
// buffers and issues S(n + 1) ahead, then dQ(n), X(n + 1).
//
// A unit's own tile has 128 rows; a step takes W rows of the other side: 128 at d = 128
// (one block per SM), 64 at d = 64, where the products are small and what counts is to
// hide the hand-overs between tensor core and rows: half the tensor memory, so that two
// blocks share an SM.
//
// Roles: warps 0 .. W/8 - 1 the rows (thread = TMEM lane x 32 columns), then a warp for
// the TMA loads, one for TMEM allocation and the MMAs, and two that form delta ahead of
// the rows (DQ; idle in DKV).
//
// 8 x 16 heads x 2048 x 64, w = 64, 4 sinks: 145 us (113 without sinks); 2 x 16 heads
// (4 key/value) x 8192 x 128, w = 1024: 512 us, 630 TFLOP/s of 10 d per visible pair, the
// least a backward needs. The rows bound it (a step of 128 x 128 pairs takes them about
// 3200 cycles, while the tensor pipe is busy 42% of DQ and 52% of DKV): loads from tensor
// memory, masks, exponentials, two conversions. Outputs by TMA from shared memory, and
// prefetching the next unit's own tiles into L2, made no difference or cost time.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "sink.cuh"
#include "sink_tc.cuh"
#include "sink_walk.cuh"
#include "tcgen05_heads.cuh"
#include "tma_host.h"

namespace based {
namespace {

using namespace tc;

constexpr int C = kOwnRows;                  // rows of a unit's own tile

template <int D, bool DKV>
struct BwdLayout {
    static constexpr int W = D;                              // rows of a step: 64 or 128
    static constexpr int CG = W / 32;                        // column groups: row warps per lane quadrant
    static constexpr int ROW_WARPS = 4 * CG;
    static constexpr int THREADS = (ROW_WARPS + 4) * 32;
    static constexpr int BLOCKS_PER_SM = W == 64 ? 2 : 1;
    // Registers per thread: 80 (384 threads, twice) or 96 (640) at launch. At d = 64 the four
    // control warps hand some to the rows: 2 x 88 + 64 = 3 x 80.
    static constexpr int ROW_REGS = W == 64 ? 88 : 0;
    [[maybe_unused]] static constexpr int CONTROL_REGS = 64;
    static constexpr uint32_t BLOCK = C * 128, RBLOCK = W * 128;   // 64 columns, 128-byte swizzle: own, ring
    static constexpr uint32_t TILE = C * D * 2, RTILE = W * D * 2;
    static constexpr int STAGES = D == 64 ? 4 : 2;           // ring stages of the other side's two tiles
    static constexpr uint32_t OFF_OWN = 0;                   // Q, dY (DQ) or K, V (DKV)
    static constexpr uint32_t OFF_A = OFF_OWN + 2 * TILE;              // [STAGES]: K (DQ) or Q (DKV)
    static constexpr uint32_t OFF_B = OFF_A + STAGES * RTILE;          // [STAGES]: V (DQ) or dY (DKV)
    static constexpr uint32_t OFF_ROW = OFF_B + STAGES * RTILE;        // DKV [STAGES][2][W]: -lse log2 e, delta
    // DQ, each by parity of their units: -lse log2 e and delta [2][128] from the delta warps;
    // partial deltas of a sweep [CG][128].
    static constexpr uint32_t OFF_DELTA = OFF_ROW + STAGES * 2 * W * 4;
    static constexpr uint32_t OFF_SCAN = OFF_DELTA + (DKV ? 0 : 2 * 2 * C * 4);
    static constexpr uint32_t OFF_HEAD = OFF_SCAN + (DKV ? 0 : 2 * CG * C * 4);   // [STAGES] Head
    static constexpr uint32_t OFF_BAR = OFF_HEAD + STAGES * 32;
    static constexpr uint32_t SMEM_BYTES = OFF_BAR + 512 + 1024;
    static_assert(STAGES <= 4, "barriers of the ring");
    static_assert(BLOCKS_PER_SM * (SMEM_BYTES + 1024) <= 228 * 1024, "shared memory");
    // DKV: S, X, dV, dK. DQ: two S, X, dQ.
    static constexpr uint32_t COL_S = 0, COL_X = DKV ? W : 2 * W;
    static constexpr uint32_t COL_ACC = DKV ? 2 * W : 3 * W; // DKV: dV, then dK at + D
    static constexpr uint32_t TMEM_COLS = 512 / BLOCKS_PER_SM;
    static_assert(COL_ACC + (DKV ? 2 : 1) * D <= TMEM_COLS, "tensor memory");
};

enum {
    GB_OWNF = 0,              // TMA: own tiles landed
    GB_OWNE = 2,              // MMA commit: own tiles no longer read
    GB_AF = 4,                // [4] TMA: ring tile A (K or Q) landed
    GB_AE = 8,                // [4] MMA commit: read
    GB_BF = 12,               // [4] ring tile B (V or dY)
    GB_BE = 16,               // [4]
    GB_SF = 20,               // [2] MMA commit: S ready (DQ: buffer of the step's parity)
    GB_XF = 22,               // MMA commit: X ready
    GB_PF,                    // DKV row warps: P written
    GB_DF,                    // row warps: dS written
    GB_ACCF,                  // MMA commit: the unit's accumulators complete
    GB_ACCE,                  // row warps: accumulators read out
    GB_RED,                   // DQ row warps: partial deltas of the sweep written
    GB_DLF,                   // [2] DQ delta warps: a unit's -lse log2 e and delta written
    GB_DLE = GB_DLF + 2,      // [2] DQ row warps: read
    GB_NUM = GB_DLE + 2
};

struct BwdParams {
    const int64_t* lengths;
    const float* lse;
    View q, k, v, y, dy, dq, dk, dv;
    float* nl2;                              // [B Hq][npad]: -lse log2 e
    float* delta;                            // [B Hq][npad]
    float* partial;
    unsigned* status;
    SinkSplit sp;
    FastDiv by_bhq, by_bhkv, by_hq, by_hkv, by_group;
    int wide_dq, wide_dk, wide_dv;           // 32-byte rows
    int B, Hq, Hkv, N, w, n_sink, sk, nt, npad, units;
    float c, scale;
    unsigned debug;
};

struct BwdCtx {
    uint32_t sbase;
    uint64_t* bars;
    volatile int* abort_flag;
    volatile int* redo;                      // some row came out non-finite
    unsigned* status;
};

__device__ __forceinline__ bool gwait(const BwdCtx& cx, int bar, uint32_t parity) {
    return mbar_wait(&cx.bars[bar], parity, cx.abort_flag, cx.status);
}
__device__ __forceinline__ bool gwait_joint(const BwdCtx& cx, int bar, uint32_t parity) {
    return mbar_wait_joint(&cx.bars[bar], parity, cx.abort_flag, cx.status);
}
__device__ __forceinline__ bool gwait_warp(const BwdCtx& cx, int bar, uint32_t parity) {
    return mbar_wait_warp(&cx.bars[bar], parity, cx.abort_flag, cx.status);
}
// After an abort: wait (bounded) for this thread's own last asynchronous work.
__device__ __forceinline__ void gdrain(const BwdCtx& cx, int bar, uint32_t parity) {
    if (!*cx.abort_flag || bar < 0) return;
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait(&cx.bars[bar], parity) && global_ns() - t0 < kWaitLimitNs) {}
}

__device__ __forceinline__ __nv_bfloat16* row_ptr(const View& v, int b, int h, int n) {
    return row_of<__nv_bfloat16>(v, b, h, n);
}

// ------------------------------------------------------------------ TMA loads (the first warp after the rows)
struct BwdMaps {
    const CUtensorMap *own0, *own1, *a, *b, *a_sink, *b_sink;
};

template <int D, bool DKV, typename Walk>
__device__ __forceinline__ void bwd_load(const BwdCtx& cx, const BwdParams& p, const BwdMaps& m) {
    using L = BwdLayout<D, DKV>;
    int g = 0, nu = 0, last = -1;
    uint32_t lastp = 0;
    Walk wk;
    for (wk.start(p, blockIdx.x); wk.u < p.units;) {
        if (!DKV) seq_len(p.lengths, wk.b, p.N, p.status);   // reports a length out of range
        if (nu >= 1 && !gwait(cx, GB_OWNE, (nu - 1) & 1)) { gdrain(cx, last, lastp); return; }
        mbar_expect_tx(&cx.bars[GB_OWNF], 2 * L::TILE);
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
            const uint32_t o = cx.sbase + L::OFF_OWN + h * L::BLOCK;
            tma_load_4d(o, m.own0, &cx.bars[GB_OWNF], 64 * h, wk.own, wk.own_head(), wk.b);
            tma_load_4d(o + L::TILE, m.own1, &cx.bars[GB_OWNF], 64 * h, wk.own, wk.own_head(), wk.b);
        }
        last = GB_OWNF, lastp = nu & 1;
        ++nu;
        for (bool final = false; !final; ++g) {
            const int st = g % L::STAGES;
            const uint32_t ph = (g / L::STAGES) & 1;
            const bool sink = wk.sink();
            const uint32_t blk = sink ? p.sk * 128u : L::RBLOCK;
            const int row = wk.ring_row(), head = wk.ring_head();
            const uint32_t head_at = cx.sbase + L::OFF_HEAD + st * (uint32_t)sizeof(Head);
            final = wk.last();
            const bool end = final && wk.u + gridDim.x >= p.units;
            const int flags = (final ? Head::kLast : 0) | (sink ? Head::kSink : 0) | (end ? Head::kEnd : 0) | wk.sweep();
            if (g >= L::STAGES && !gwait(cx, GB_AE + st, ph ^ 1)) { gdrain(cx, last, lastp); return; }
            st_shared_v4(head_at, make_uint4(wk.own, row, wk.len, flags));
            st_shared_v4(head_at + 16, make_uint4(wk.b, wk.own_head(), wk.tag(), 0));
            mbar_expect_tx(&cx.bars[GB_AF + st], blk * (D / 64) + (DKV ? 2 * L::W * 4 : 0));
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
                tma_load_4d(cx.sbase + L::OFF_A + st * L::RTILE + h * blk, sink ? m.a_sink : m.a, &cx.bars[GB_AF + st],
                            64 * h, row, head, wk.b);
            if constexpr (DKV) {                             // with Q: released with it, after the last rows read them
                const size_t vec = ((size_t)wk.b * p.Hq + head) * p.npad + row;
                const uint32_t rows = cx.sbase + L::OFF_ROW + st * 2 * L::W * 4;
                bulk_load(rows, p.nl2 + vec, L::W * 4, &cx.bars[GB_AF + st]);
                bulk_load(rows + L::W * 4, p.delta + vec, L::W * 4, &cx.bars[GB_AF + st]);
            }
            last = GB_AF + st, lastp = ph;
            if (g >= L::STAGES && !gwait(cx, GB_BE + st, ph ^ 1)) { gdrain(cx, last, lastp); return; }
            mbar_expect_tx(&cx.bars[GB_BF + st], blk * (D / 64));
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
                tma_load_4d(cx.sbase + L::OFF_B + st * L::RTILE + h * blk, sink ? m.b_sink : m.b, &cx.bars[GB_BF + st],
                            64 * h, row, head, wk.b);
            last = GB_BF + st, lastp = ph;
            if (!final) wk.next();
        }
        wk.start(p, wk.u + gridDim.x);
    }
    gdrain(cx, last, lastp);
}

// ------------------------------------------------------------------ MMAs (the second)
template <int D, bool DKV>
__device__ __forceinline__ void bwd_mma(const BwdCtx& cx, const BwdParams& p, uint32_t tmem) {
    using L = BwdLayout<D, DKV>;
    constexpr uint32_t id_s = idesc_bf16_f32(C, L::W, false, false), id_acc = idesc_bf16_f32(C, D, false, true);
    const uint32_t id_sink = idesc_bf16_f32(C, p.sk, false, false);
    // Descriptors of the first buffers; tiles and K steps add to their address field (16-byte units).
    const uint64_t d_own = smem_desc_sw128(cx.sbase + L::OFF_OWN, 16, 1024),
                   d_a = smem_desc_sw128(cx.sbase + L::OFF_A, 16, 1024), d_b = smem_desc_sw128(cx.sbase + L::OFF_B, 16, 1024),
                   m_a = smem_desc_sw128(cx.sbase + L::OFF_A, L::RBLOCK, 1024),
                   m_b = smem_desc_sw128(cx.sbase + L::OFF_B, L::RBLOCK, 1024),
                   m_a_sink = smem_desc_sw128(cx.sbase + L::OFF_A, p.sk * 128u, 1024);
    constexpr uint32_t TILE16 = L::TILE >> 4, BLOCK16 = L::BLOCK >> 4, RTILE16 = L::RTILE >> 4, RBLOCK16 = L::RBLOCK >> 4;
    bool ok = true;
    int flags = 0, next = 0;                 // of the current step, of the one whose S was issued last
    // D = own0 A^T (which 0: S; reads the step's header first) or own1 B^T (1: X) of ring step g.
    const auto pair = [&](int which, int g) {
        const int st = g % L::STAGES;
        ok = ok && gwait_warp(cx, (which ? GB_BF : GB_AF) + st, (g / L::STAGES) & 1);
        if (!ok) return;
        if (!which) next = (int)__float_as_uint(ld_shared_f32(cx.sbase + L::OFF_HEAD + st * (uint32_t)sizeof(Head) + 12));
        tc_fence_after();
        const bool sink = !DKV && (next & Head::kSink);
        const uint64_t a = d_own + which * TILE16, b = (which ? d_b : d_a) + st * RTILE16;
        const uint32_t dst = tmem + (which ? L::COL_X : L::COL_S + (DKV ? 0 : L::W * (g & 1)));
        if (elect_one()) {
            if (sink) {
                for (int k = 0; k < D / 16; ++k)
                    mma_bf16(dst, a + (k >> 2) * BLOCK16 + (k & 3) * 2, b + (k >> 2) * p.sk * 8 + (k & 3) * 2, id_sink, k > 0);
            } else {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_bf16(dst, a + ((k >> 2) * BLOCK16 + (k & 3) * 2), b + ((k >> 2) * RBLOCK16 + (k & 3) * 2), id_s, k > 0);
            }
            mma_commit(&cx.bars[which ? GB_XF : GB_SF + (DKV ? 0 : (g & 1))]);
            if (!DKV && which) mma_commit(&cx.bars[GB_BE + st]);             // V is read by X only
            if (which && (next & Head::kLast)) mma_commit(&cx.bars[GB_OWNE]);   // S went before
        }
        __syncwarp();
    };
    // acc += (operand of the rows at column `src`) (ring tile as K rows).
    const auto product = [&](uint32_t acc, uint32_t src, uint64_t b, bool sink, bool first) {
        if (sink) {
            for (int k = 0; k < p.sk / 16; ++k)
                mma_bf16_ts(tmem + acc, tmem + src + 16 * k, b + k * 128, id_acc, (!first || k > 0) ? 1u : 0u);
        } else {
            mma_bf16_ts(tmem + acc, tmem + src, b, id_acc, first ? 0u : 1u);
#pragma unroll
            for (int k = 1; k < L::W / 16; ++k) mma_bf16_ts(tmem + acc, tmem + src + 16 * k, b + k * 128, id_acc, 1u);
        }
    };
    int g = 0, nu = 0;                       // steps, finished units
    ok = gwait_warp(cx, GB_OWNF, 0);
    pair(0, 0);
    pair(1, 0);
    while (ok) {
        flags = next;
        const int st = g % L::STAGES;
        const bool sink = flags & Head::kSink, final = flags & Head::kLast, more = !(flags & Head::kEnd);
        const bool first = flags & Head::kFirst;
        if constexpr (DKV) {
            ok = gwait_warp(cx, GB_PF, g & 1);
            if (ok && first && nu > 0) ok = gwait_warp(cx, GB_ACCE, (nu - 1) & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                product(L::COL_ACC, L::COL_S, m_b + st * RTILE16, false, first);         // dV += P dY
                mma_commit(&cx.bars[GB_BE + st]);
            }
            __syncwarp();
            if (!final) pair(0, g + 1);      // the next unit's S waits for its own tiles, below
            ok = ok && gwait_warp(cx, GB_DF, g & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                product(L::COL_ACC + D, L::COL_X, m_a + st * RTILE16, false, first);     // dK += dS Q
                mma_commit(&cx.bars[GB_AE + st]);
                if (final) mma_commit(&cx.bars[GB_ACCF]);
            }
            __syncwarp();
        } else {
            if (!final) pair(0, g + 1);
            ok = ok && gwait_warp(cx, GB_DF, g & 1);
            if (ok && first && nu > 0) ok = gwait_warp(cx, GB_ACCE, (nu - 1) & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                if (!(flags & Head::kScan))
                    product(L::COL_ACC, L::COL_X, (sink ? m_a_sink : m_a) + st * RTILE16, sink, first);   // dQ += dS K
                mma_commit(&cx.bars[GB_AE + st]);
                if (final) mma_commit(&cx.bars[GB_ACCF]);
            }
            __syncwarp();
        }
        if (final) {
            ++nu;
            if (!more) break;
            ok = gwait_warp(cx, GB_OWNF, nu & 1);
            pair(0, g + 1);
        }
        pair(1, g + 1);
        ++g;
    }
    // Every MMA has completed: the last unit's accumulators are the last commit.
    if (ok) gwait_warp(cx, GB_ACCF, (nu - 1) & 1);
    else if (g > 0) gdrain(cx, GB_AE + (g - 1) % L::STAGES, ((g - 1) / L::STAGES) & 1);
}

// ------------------------------------------------------------------ delta (DQ: the third and fourth)

// -lse log2 e and delta = dy . y of a unit's rows, ahead of the row warps and in their
// stead: taken by them, the loads' latency came to 5000 of a unit's 18000 cycles (8 x 16
// heads x 2048 x 64, w = 64: the backward 150 -> 138 us; 2 x 16 heads x 8192 x 128,
// w = 1024: 561 -> 513). Warp `half` takes 64 rows, D / 8 lanes each, so that a load
// reads whole lines.
template <int D>
__device__ __forceinline__ void dq_delta(const BwdCtx& cx, const BwdParams& p, int half, int lane) {
    using L = BwdLayout<D, false>;
    constexpr int LPR = D / 8, STEP = 32 / LPR, BATCH = 4;   // lanes per row, rows per load, loads in flight
    int nu = 0;                              // units so far, but for those with a sweep of their own
    for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
        DqWalk<L::W> wk;
        wk.start(p, u);
        if (wk.scan) continue;
        const int r0 = 64 * half, buf = nu & 1;
        const size_t row = (size_t)wk.b * p.Hq + wk.h;
        float nl[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int i = wk.own + r0 + 32 * x + lane;
            nl[x] = i < wk.len ? -p.lse[row * p.N + i] * kLog2e : 0.f;
        }
        if (nu >= 2 && !gwait_warp(cx, GB_DLE + buf, ((nu >> 1) - 1) & 1)) return;
        const uint32_t red = cx.sbase + L::OFF_DELTA + buf * 2 * C * 4 + r0 * 4;
        for (int r = 0; r < 64; r += BATCH * STEP) {
            uint4 x[BATCH], z[BATCH];
#pragma unroll
            for (int q = 0; q < BATCH; ++q) {
                x[q] = z[q] = make_uint4(0, 0, 0, 0);
                const int i = wk.own + r0 + r + q * STEP + lane / LPR;
                if (i < wk.len) {
                    x[q] = __ldg(reinterpret_cast<const uint4*>(row_ptr(p.dy, wk.b, wk.h, i)) + lane % LPR);
                    z[q] = __ldg(reinterpret_cast<const uint4*>(row_ptr(p.y, wk.b, wk.h, i)) + lane % LPR);
                }
            }
#pragma unroll
            for (int q = 0; q < BATCH; ++q) {
                float d = dot16(x[q], z[q], 0.f, static_cast<const __nv_bfloat16*>(nullptr));
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
                if (lane % LPR == 0) st_shared_f32(red + (C + r + q * STEP + lane / LPR) * 4, d);
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) st_shared_f32(red + (32 * x + lane) * 4, nl[x]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&cx.bars[GB_DLF + buf]);
#pragma unroll
        for (int x = 0; x < 2; ++x) {                        // for DKV
            const size_t at = row * p.npad + wk.own + r0 + 32 * x + lane;
            p.nl2[at] = nl[x];
            p.delta[at] = ld_shared_f32(red + (C + 32 * x + lane) * 4);
        }
        __syncwarp();
        ++nu;
    }
}

// ------------------------------------------------------------------ rows (the first warps)

// p = 2^(s c + n) of 32 columns (n: one value per column in shared memory, or one for the row).
__device__ __forceinline__ void add_scaled(float* s, float c, float n0, float n1, float n2, float n3) {
    asm("{\n\t.reg .b64 a, b, c, d, e;\n\t"
        "mov.b64 a, {%0, %1};\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "mov.b64 c, {%4, %4};\n\t"
        "mov.b64 d, {%5, %6};\n\t"
        "mov.b64 e, {%7, %8};\n\t"
        "fma.rn.f32x2 a, a, c, d;\n\t"
        "fma.rn.f32x2 b, b, c, e;\n\t"
        "mov.b64 {%0, %1}, a;\n\t"
        "mov.b64 {%2, %3}, b;\n\t}"
        : "+f"(s[0]), "+f"(s[1]), "+f"(s[2]), "+f"(s[3])
        : "f"(c), "f"(n0), "f"(n1), "f"(n2), "f"(n3));
}
// x = p (x - d) for two columns.
__device__ __forceinline__ void dscore(float& x0, float& x1, float p0, float p1, float d0, float d1) {
    asm("{\n\t.reg .b64 x, p, d;\n\t"
        "mov.b64 x, {%0, %1};\n\t"
        "mov.b64 p, {%2, %3};\n\t"
        "mov.b64 d, {%4, %5};\n\t"
        "sub.rn.f32x2 x, x, d;\n\t"
        "mul.rn.f32x2 x, x, p;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "+f"(x0), "+f"(x1)
        : "f"(p0), "f"(p1), "f"(d0), "f"(d1));
}
__device__ __forceinline__ void ld_shared_f4(uint32_t a, float* v) {
    const uint4 x = ld_shared_v4(a);
    v[0] = __uint_as_float(x.x), v[1] = __uint_as_float(x.y);
    v[2] = __uint_as_float(x.z), v[3] = __uint_as_float(x.w);
}

// Writes 32 columns as a bf16 A operand over the scores they come from: K step k (16
// columns) at the first 8 of its 16 TMEM columns.
__device__ __forceinline__ void put32(uint32_t taddr, const float* x) {
    uint32_t b[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) b[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    tmem_st8(taddr, b);
    tmem_st8(taddr + 16, b + 8);
}

// Rows [r0, r1) of a ring tile (W rows of D columns in blocks of `blk` bytes) set to zero
// by all row threads, 32 bytes of a block each.
template <int D, int W>
__device__ __forceinline__ void zero_rows(uint32_t tile, uint32_t blk, int r0, int r1, int r, int cg) {
    const int row = r % W, part = r / W * (W / 32) + cg;
    if (row >= r0 && row < r1) {
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
            st_shared_v4(tile + h * blk + row * 128 + 32 * part, make_uint4(0, 0, 0, 0));
            st_shared_v4(tile + h * blk + row * 128 + 32 * part + 16, make_uint4(0, 0, 0, 0));
        }
    }
    fence_proxy_async_smem();
    __syncwarp();
}

// Reads this thread's share (columns n cg ..) of an accumulator row, scales it and hands
// over 16 columns at a time. NaN where one of them is not finite, else 0.
template <int N, typename F>
__device__ __forceinline__ float read_out(uint32_t taddr, int cg, float scale, F&& put) {
    float odd = 0.f;
#pragma unroll
    for (int q = 0; q < N / 16; ++q) {
        float o[16];
        tmem_ld16(taddr + N * cg + 16 * q, o);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            o[e] *= scale;
            odd = fmaf(o[e], 0.f, odd);
        }
        put(N * cg + 16 * q, o);
        __syncwarp();
    }
    return odd;
}

template <int D>
__device__ __forceinline__ void dq_rows(const BwdCtx& cx, const BwdParams& p, uint32_t tmem, int cg, int wq, int lane) {
    using L = BwdLayout<D, false>;
    constexpr int W = L::W, CG = L::CG, SHARE = D / CG;      // SHARE: channels of a row per thread
    const int r = wq * 32 + lane, c0 = 32 * cg;
    const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    int nu = 0, nd = 0, ns = 0;                              // units; with delta from its warps; from a sweep
    bool first = true;
    float nl = 0.f, delta = 0.f;                             // -lse log2 e and delta of the row
    for (int g = 0;; ++g) {
        const int st = g % L::STAGES;
        if (!gwait_joint(cx, GB_AF + st, (g / L::STAGES) & 1)) return;
        const uint32_t head = cx.sbase + L::OFF_HEAD + st * (uint32_t)sizeof(Head);
        const uint4 hd = ld_shared_v4(head);
        const int i0 = hd.x, len = hd.z, i = i0 + r;
        const bool sink = hd.w & Head::kSink, last = hd.w & Head::kLast, live = i < len;
        const bool scan = hd.w & Head::kScan;
        if (first) {
            if (scan) {
                const uint4 hb = ld_shared_v4(head + 16);
                nl = live ? -p.lse[((size_t)hb.x * p.Hq + hb.y) * p.N + i] * kLog2e : 0.f;
                delta = 0.f;
            } else {
                if (!gwait_joint(cx, GB_DLF + (nd & 1), (nd >> 1) & 1)) return;
                const uint32_t at = cx.sbase + L::OFF_DELTA + (nd & 1) * 2 * C * 4 + r * 4;
                nl = ld_shared_f32(at);
                delta = ld_shared_f32(at + C * 4);
                __syncwarp();
                if (lane == 0) mbar_arrive(&cx.bars[GB_DLE + (nd & 1)]);
                ++nd;
            }
        }
        const int j0 = hd.y;
        uint32_t vis = ~0u;
        if (sink || j0 + W > i0 + 1 || j0 < i0 + C - p.w) {
            const int hi = (sink ? p.n_sink : i - j0 + 1) - c0, lo = (sink ? 0 : i - p.w + 1 - j0) - c0;
            vis = low_bits(hi) & (~low_bits(lo) | low_bits((j0 == 0 ? p.n_sink : 0) - c0));
        }
        const WordMask mask(vis);
        const bool any = mask.kind != WordMask::kNone;       // for some row of this warp
        if (!gwait_joint(cx, GB_SF + (g & 1), (g >> 1) & 1)) return;
        tc_fence_after();
        float pr[32];
        if (any) {
            tmem_ld32(tl + L::COL_S + W * (g & 1) + c0, pr);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; e += 4) add_scaled(pr + e, p.c, nl, nl, nl, nl);
#pragma unroll
            for (int e = 0; e < 32; ++e) pr[e] = ex2(pr[e]);
            mask.apply(pr, 0.f);
        }
        // K rows that no dS may meet: padding in the tile of the sequence's end, tokens
        // after the sinks in their block.
        const int k0 = sink ? p.n_sink : len - j0, k1 = sink ? p.sk : min(W, p.N - j0);
        if ((sink || last) && k0 < k1)
            zero_rows<D, W>(cx.sbase + L::OFF_A + st * L::RTILE, sink ? p.sk * 128u : L::RBLOCK, k0, k1, r, cg);
        if (!gwait_joint(cx, GB_XF, g & 1)) return;
        tc_fence_after();
        {
            float x[32];
            if (any) {
                tmem_ld32(tl + L::COL_X + c0, x);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; e += 2)
                    dscore(x[e], x[e + 1], pr[e], pr[e + 1], scan ? 0.f : delta, scan ? 0.f : delta);
                mask.apply(x, 0.f);
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = 0.f;
            }
            if (scan) {                                      // p dP, kept in fp32
                float t0 = 0.f, t1 = 0.f;
#pragma unroll
                for (int e = 0; e < 32; e += 2) add_pair(t0, t1, x[e], x[e + 1]);
                delta += t0 + t1;                            // of this column group, until published
                if (hd.w & Head::kScanEnd) {                 // summed over the groups, and handed on to DKV
                    const uint32_t red = cx.sbase + L::OFF_SCAN + (ns & 1) * CG * C * 4 + r * 4;
                    st_shared_f32(red + cg * C * 4, live ? delta : 0.f);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&cx.bars[GB_RED]);
                    if (!gwait_joint(cx, GB_RED, ns++ & 1)) return;
                    delta = 0.f;
#pragma unroll
                    for (int q = 0; q < CG; ++q) delta += ld_shared_f32(red + q * C * 4);
                    if (cg == 0) {
                        const uint4 hb = ld_shared_v4(head + 16);
                        const size_t row = ((size_t)hb.x * p.Hq + hb.y) * p.npad + i;
                        p.nl2[row] = nl;
                        p.delta[row] = delta;
                    }
                }
            } else {
                put32(tl + L::COL_X + c0, x);
            }
        }
        // The header may be overwritten once every row warp is through with the step.
        const uint4 hb = last ? ld_shared_v4(head + 16) : make_uint4(0, 0, 0, 0);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&cx.bars[GB_DF]);
        first = last;
        if (!last) continue;
        if (!gwait_joint(cx, GB_ACCF, nu & 1)) return;
        tc_fence_after();
        __nv_bfloat16* out = row_ptr(p.dq, hb.x, hb.y, i);
        const float odd = read_out<SHARE>(tl + L::COL_ACC, cg, p.scale, [&](int col, const float* o) {
            if (i < p.N)
                store16(out + col, live ? pack_bf16x8(o) : make_uint4(0, 0, 0, 0),
                        live ? pack_bf16x8(o + 8) : make_uint4(0, 0, 0, 0), p.wide_dq);
        });
        if (live && odd != 0.f) *cx.redo = 1;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&cx.bars[GB_ACCE]);
        ++nu;
        if (hd.w & Head::kEnd) return;
    }
}

template <int D>
__device__ __forceinline__ void dkv_rows(const BwdCtx& cx, const BwdParams& p, uint32_t tmem, int cg, int wq, int lane) {
    using L = BwdLayout<D, true>;
    constexpr int W = L::W, SHARE = D / L::CG;               // SHARE: channels of a row per thread
    const int r = wq * 32 + lane, c0 = 32 * cg;
    const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    int nu = 0;
    for (int g = 0;; ++g) {
        const int st = g % L::STAGES;
        const uint32_t ph = (g / L::STAGES) & 1;
        if (!gwait_joint(cx, GB_AF + st, ph)) return;
        const uint32_t head = cx.sbase + L::OFF_HEAD + st * (uint32_t)sizeof(Head);
        const uint4 hd = ld_shared_v4(head), hb = ld_shared_v4(head + 16);
        const int j0 = hd.x, i0 = hd.y, len = hd.z, j = j0 + r;
        const bool last = hd.w & Head::kLast, chunk = (int)hb.z >= 0;
        // Visible queries of this key: [j, j + w) in a band unit, [j + w, ..) for a sink in
        // a chunk; none past the sequence's end.
        uint32_t vis = ~0u;
        if (chunk || i0 < j0 + C || i0 + W > j0 + p.w || i0 + W > len) {
            const QueryRange q(chunk, j, len, p.w, p.n_sink);
            vis = low_bits(q.end - i0 - c0) & ~low_bits(q.from - i0 - c0);
        }
        const WordMask mask(vis);
        const bool any = mask.kind != WordMask::kNone;       // for some row of this warp
        if (!gwait_joint(cx, GB_SF, g & 1)) return;
        tc_fence_after();
        const uint32_t rows = cx.sbase + L::OFF_ROW + st * 2 * W * 4 + 4 * c0;
        float pr[32];
        if (any) {
            tmem_ld32(tl + L::COL_S + c0, pr);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                float n[4];
                ld_shared_f4(rows + 4 * e, n);
                add_scaled(pr + e, p.c, n[0], n[1], n[2], n[3]);
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) pr[e] = ex2(pr[e]);
            mask.apply(pr, 0.f);
        } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) pr[e] = 0.f;
        }
        put32(tl + L::COL_S + c0, pr);
        // Rows of Q and dY that no weight may meet: padding in the tile of the sequence's end.
        if (i0 + W > len && len < p.N) {
            if (!gwait_joint(cx, GB_BF + st, ph)) return;
            zero_rows<D, W>(cx.sbase + L::OFF_A + st * L::RTILE, L::RBLOCK, len - i0, W, r, cg);
            zero_rows<D, W>(cx.sbase + L::OFF_B + st * L::RTILE, L::RBLOCK, len - i0, W, r, cg);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&cx.bars[GB_PF]);
        if (!gwait_joint(cx, GB_XF, g & 1)) return;
        tc_fence_after();
        {
            float x[32];
            if (any) {
                tmem_ld32(tl + L::COL_X + c0, x);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    float d[4];
                    ld_shared_f4(rows + W * 4 + 4 * e, d);
                    dscore(x[e], x[e + 1], pr[e], pr[e + 1], d[0], d[1]);
                    dscore(x[e + 2], x[e + 3], pr[e + 2], pr[e + 3], d[2], d[3]);
                }
                mask.apply(x, 0.f);
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = 0.f;
            }
            put32(tl + L::COL_X + c0, x);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&cx.bars[GB_DF]);
        if (!last) continue;
        if (!gwait_joint(cx, GB_ACCF, nu & 1)) return;
        tc_fence_after();
        // Sink rows go to partials (slot 0: the sink tile's band unit, 1 + c: chunk c).
        const int b = hb.x, hk = hb.y;
        const bool zero = j >= len;
        float odd = 0.f;
        if (p.sp.chunks > 0 && j0 == 0 && wq * 32 < p.n_sink) {   // the other warps hold no sink
            float* part = p.partial + sink_partial_offset(p.sp, b * p.Hkv + hk, (int)hb.z + 1, D) + (size_t)r * D;
            const auto put = [&](float* to, const float* o) {
                if (r >= p.n_sink || j >= p.N) return;
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    *reinterpret_cast<float4*>(to + e) =
                        zero ? make_float4(0, 0, 0, 0) : make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            };
            odd += read_out<SHARE>(tl + L::COL_ACC, cg, 1.0f,
                                   [&](int col, const float* o) { put(part + (size_t)p.sp.rows * D + col, o); });
            odd += read_out<SHARE>(tl + L::COL_ACC + D, cg, p.scale, [&](int col, const float* o) { put(part + col, o); });
        }
        if (!chunk) {
            const bool store = j < p.N && !(p.sp.chunks > 0 && j < p.n_sink);
            const auto put = [&](__nv_bfloat16* to, const float* o, bool wide) {
                if (store)
                    store16(to, zero ? make_uint4(0, 0, 0, 0) : pack_bf16x8(o),
                            zero ? make_uint4(0, 0, 0, 0) : pack_bf16x8(o + 8), wide);
            };
            __nv_bfloat16* ov = row_ptr(p.dv, b, hk, j);
            odd += read_out<SHARE>(tl + L::COL_ACC, cg, 1.0f, [&](int col, const float* o) { put(ov + col, o, p.wide_dv); });
            __nv_bfloat16* ok = row_ptr(p.dk, b, hk, j);
            odd += read_out<SHARE>(tl + L::COL_ACC + D, cg, p.scale,
                                   [&](int col, const float* o) { put(ok + col, o, p.wide_dk); });
        }
        if (!zero && odd != 0.f) *cx.redo = 1;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&cx.bars[GB_ACCE]);
        ++nu;
        if (hd.w & Head::kEnd) return;
    }
}

// Non-finite rows of the block's units, again from their definition (see GradRow). A row is
// computed from what -lse log2 e and delta the workspace holds, which no hidden pair reaches.
template <int D>
__device__ __noinline__ void dq_redo(const BwdParams& p, int warp) {
    using L = BwdLayout<D, false>;
    for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
        DqWalk<L::W> wk;
        wk.start(p, u);
        const size_t at = ((size_t)wk.b * p.Hq + wk.h) * p.npad;
        bool checked = false;
        for (int i = wk.own + warp; i < min(wk.own + C, wk.len); i += L::ROW_WARPS) {
            __nv_bfloat16* out = row_ptr(p.dq, wk.b, wk.h, i);
            if (!odd_row<D>(out)) continue;
            if (!checked && !odd_hidden_keys<D>(row_of<const __nv_bfloat16>(p.k, wk.b, wk.hk, 0), p.k.sn, wk.own, C, wk.len,
                                                wk.lo * L::W, p.w, p.n_sink, 0))
                break;
            checked = true;
            const GradRow<D> x =
                sink_exact_dq<__nv_bfloat16, D>(p, wk.b, wk.h, wk.hk, i, p.c, p.nl2 + at, 1.0f, p.delta + at);
            put_row<D>(out, x.a, p.scale);
        }
    }
}
template <int D>
__device__ __noinline__ void dkv_redo(const BwdParams& p, int warp) {
    using L = BwdLayout<D, true>;
    for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
        KvWalk<L::W> first;
        first.start(p, u);
        const int b = first.b, hk = first.hk;
        bool checked = false;
        for (int j = first.own + warp; j < min(first.own + C, first.len); j += L::ROW_WARPS) {
            const bool sink = p.sp.chunks > 0 && j < p.n_sink;       // a row of the unit's partials
            if (first.chunk >= 0 && !sink) break;
            float* pk = p.partial + sink_partial_offset(p.sp, b * p.Hkv + hk, first.chunk + 1, D) + (size_t)j * D;
            float* pv = pk + (size_t)p.sp.rows * D;
            const bool odd = sink ? odd_row<D>(pk) || odd_row<D>(pv)
                                  : odd_row<D>(row_ptr(p.dk, b, hk, j)) || odd_row<D>(row_ptr(p.dv, b, hk, j));
            if (!odd) continue;
            if (!checked &&
                !odd_hidden_queries<D, __nv_bfloat16>(p, b, hk * p.sp.group, p.sp.group, first.chunk >= 0, first.own, C,
                                                      first.len, first.t0 * L::W, (first.t0 + first.span) * L::W))
                break;
            checked = true;
            GradRow<D> x;
            for (KvWalk<L::W> wk = first;; wk.next()) {
                const QueryRange q(wk.chunk >= 0, j, wk.len, p.w, p.n_sink);
                sink_exact_dkv<__nv_bfloat16, D>(x, p, b, wk.h, hk, j, max(wk.ring_row(), q.from),
                                                 min(wk.ring_row() + L::W, q.end), p.c, p.nl2, 1.0f, p.delta, p.npad);
                if (wk.last()) break;
            }
            if (sink) {
                put_row<D>(pk, x.a, p.scale);
                put_row<D>(pv, x.b, 1.0f);
            } else {
                put_row<D>(row_ptr(p.dk, b, hk, j), x.a, p.scale);
                put_row<D>(row_ptr(p.dv, b, hk, j), x.b, 1.0f);
            }
        }
    }
}

template <int D, bool DKV>
__global__ void __launch_bounds__((BwdLayout<D, DKV>::THREADS), (BwdLayout<D, DKV>::BLOCKS_PER_SM))
sink_bwd_tc_kernel(const __grid_constant__ CUtensorMap own0, const __grid_constant__ CUtensorMap own1,
                   const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                   const __grid_constant__ CUtensorMap ma_sink, const __grid_constant__ CUtensorMap mb_sink,
                   const __grid_constant__ BwdParams p) {
    using L = BwdLayout<D, DKV>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    unsigned char* smem = smem_raw + (sbase - raw);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_BAR + 8 * GB_NUM);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_BAR + 8 * GB_NUM + 4);
    const BwdCtx cx{sbase, bars, abort_flag, abort_flag + 1, p.status};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int b = 0; b < GB_NUM; ++b)
            mbar_init(&bars[b], b == GB_PF || b == GB_DF || b == GB_ACCE || b == GB_RED || b >= GB_DLE ? L::ROW_WARPS : b >= GB_DLF ? 2 : 1);
        *abort_flag = 0;
        *cx.redo = 0;
        mbar_fence_init();
    }
    if (warp == L::ROW_WARPS + 1) tmem_alloc(tmem_slot, L::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();                                  // inputs and workspace may come from earlier kernels
    using Walk = typename std::conditional<DKV, KvWalk<L::W>, DqWalk<L::W>>::type;
    if (warp >= L::ROW_WARPS) {
        if constexpr (L::ROW_REGS > 0) reg_dec<L::CONTROL_REGS>();
        if (warp == L::ROW_WARPS) {
            if (lane == 0) bwd_load<D, DKV, Walk>(cx, p, BwdMaps{&own0, &own1, &ma, &mb, &ma_sink, &mb_sink});
        } else if (warp == L::ROW_WARPS + 1) {
            if (!(p.debug & DEBUG_SKIP_MMA)) bwd_mma<D, DKV>(cx, p, tmem);
        } else if constexpr (!DKV) {
            dq_delta<D>(cx, p, warp - L::ROW_WARPS - 2, lane);
        }
    } else {
        if constexpr (L::ROW_REGS > 0) reg_inc<L::ROW_REGS>();
        if constexpr (DKV) dkv_rows<D>(cx, p, tmem, warp >> 2, warp & 3, lane);
        else dq_rows<D>(cx, p, tmem, warp >> 2, warp & 3, lane);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == L::ROW_WARPS + 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, L::TMEM_COLS);
    }
    if (*cx.redo && !*abort_flag && warp < L::ROW_WARPS) {   // those that have the registers
        if constexpr (DKV) dkv_redo<D>(p, warp);
        else dq_redo<D>(p, warp);
    }
}

template <int D, bool DKV>
cudaError_t launch(const CUtensorMap& own0, const CUtensorMap& own1, const CUtensorMap& ma, const CUtensorMap& mb,
                   const CUtensorMap& mas, const CUtensorMap& mbs, const BwdParams& p, int num_sms,
                   cudaStream_t stream) {
    using L = BwdLayout<D, DKV>;
    auto kern = sink_bwd_tc_kernel<D, DKV>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(std::min(p.units, num_sms * L::BLOCKS_PER_SM)), dim3(L::THREADS), L::SMEM_BYTES, stream, own0, own1, ma, mb,
                      mas, mbs, p);
}

size_t padded_rows(int N) { return (size_t)(N + C - 1) / C * C; }

template <int D>
cudaError_t run(const SinkArgs& a, int num_sms, cudaStream_t stream) {
    BwdParams p{};
    p.lengths = a.lengths, p.lse = a.lse, p.status = a.status, p.debug = a.debug;
    p.q = a.q, p.k = a.k, p.v = a.v, p.y = a.y, p.dy = a.dy, p.dq = a.dq, p.dk = a.dk, p.dv = a.dv;
    p.B = a.B, p.Hq = a.Hq, p.Hkv = a.Hkv, p.N = a.N, p.w = a.w, p.n_sink = a.n_sink;
    p.sk = std::max(16, (a.n_sink + 15) / 16 * 16);
    p.nt = (a.N + C - 1) / C;
    p.npad = (int)padded_rows(a.N);
    p.by_bhq = FastDiv(a.B * a.Hq), p.by_bhkv = FastDiv(a.B * a.Hkv), p.by_hq = FastDiv(a.Hq);
    p.by_hkv = FastDiv(a.Hkv), p.by_group = FastDiv(a.Hq / a.Hkv);
    p.wide_dq = rows_aligned32(a.dq), p.wide_dk = rows_aligned32(a.dk), p.wide_dv = rows_aligned32(a.dv);
    p.c = a.scale * kLog2e;
    p.scale = a.scale;
    constexpr int W = BwdLayout<D, true>::W;
    p.sp = sink_split(a.Hq, a.Hkv, a.N, a.w, a.n_sink, C, W);
    const size_t vec = (size_t)a.B * a.Hq * p.npad;
    p.nl2 = static_cast<float*>(a.workspace);
    p.delta = p.nl2 + vec;
    p.partial = p.delta + vec;
    // Own tiles of 128 rows, ring tiles of W, the sink block.
    CUtensorMap mq, mk, mv, mg, rq, rk, rv, rg, mks, mvs;
    if (!heads_map(&mq, a.q, a, a.Hq, C) || !heads_map(&mg, a.dy, a, a.Hq, C) || !heads_map(&mk, a.k, a, a.Hkv, C) ||
        !heads_map(&mv, a.v, a, a.Hkv, C) || !heads_map(&rq, a.q, a, a.Hq, W) || !heads_map(&rg, a.dy, a, a.Hq, W) ||
        !heads_map(&rk, a.k, a, a.Hkv, W) || !heads_map(&rv, a.v, a, a.Hkv, W) ||
        !heads_map(&mks, a.k, a, a.Hkv, p.sk) || !heads_map(&mvs, a.v, a, a.Hkv, p.sk))
        return cudaErrorInvalidValue;
    p.units = a.B * a.Hq * p.nt;
    cudaError_t e = launch<D, false>(mq, mg, rk, rv, mks, mvs, p, num_sms, stream);
    p.units = a.B * a.Hkv * p.sp.units();
    if (e == cudaSuccess) e = launch<D, true>(mk, mv, rq, rg, rq, rg, p, num_sms, stream);
    if (e == cudaSuccess && p.sp.chunks > 0) e = launch_sink_join<__nv_bfloat16>(a, p.sp, p.partial, stream);
    return e;
}

}  // namespace

size_t sink_backward_workspace_tc(int B, int Hq, int Hkv, int N, int d, int w, int n_sink) {
    const SinkSplit sp = sink_split(Hq, Hkv, N, w, n_sink, C, d == 64 ? BwdLayout<64, true>::W : BwdLayout<128, true>::W);
    return (2 * (size_t)B * Hq * padded_rows(N) + sink_partial_offset(sp, B * Hkv, 0, d)) * sizeof(float);
}

cudaError_t launch_sink_backward_tc(const SinkArgs& a, int num_sms, cudaStream_t stream) {
    return a.d == 64 ? run<64>(a, num_sms, stream) : run<128>(a, num_sms, stream);
}

}  // namespace based
