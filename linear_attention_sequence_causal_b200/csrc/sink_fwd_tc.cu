// Prompt form of the sliding-window attention with sink tokens on the tensor cores (bf16).
//
//   y_i = sum_j p_ij v_j, p_ij = softmax_j(scale q_i.k_j) over
//   visible(i) = { j <= i : j > i - w or j < n_sink }.
// A persistent block works on two "slots" at once, each a tile of 128 queries: two
// query heads that share a key/value head where the group is even, else two
// neighbouring tiles of one head, so that one K and V tile in shared memory feeds
// both. It sweeps the 128-key tiles that either slot sees, after the sink tokens'
// own short block (n_sink rounded up to 16 keys) where the window has left them
// behind: S = Q K^T into TMEM; one thread per query row forms the weights with a
// running maximum and sum and writes them back as bf16 over S; O += P V with P read
// from TMEM. The two slots alternate: while one slot's rows compute exponentials,
// the tensor core runs the other's products.
//
// The accumulator is rescaled only when a row's maximum has grown by more than 2^8
// since the last time (any smaller growth leaves weights up to 2^8, exact in the
// same relative precision), so the row threads do it themselves. S of step j is
// committed after P V of step j - 1, so its arrival also says that O is at rest.
//
// Roles (384 threads): warps 0-3 and 4-7 the rows of slots 0 and 1 (thread = row =
// TMEM lane), warp 8 the TMA loads, warps 9 and 10 the MMAs of
// slots 0 and 1 (9 allocates TMEM; 11 idles).
// TMEM: S0, S1 (128 columns each, P over the first 64), O0, O1 (d columns each).
//
// 2 x 16 heads (4 key/value) x 16384 x 128, w = 1024, 4 sinks: 358 us, 746 TFLOP/s over
// the visible pairs (4 d each; the tiles at both edges of the window compute 1.12 times
// as many), of 1660 for a library product. A row's chain per tile (maximum, turn,
// exponentials, weights back to tensor memory) bounds it: the tensor pipe is busy 38% of
// the time. A part of the exponentials on the FMA units, 16 row warps, 64-key tiles with
// two S buffers, one speculative pass over the scores: each slower.
#include <algorithm>
#include <limits>

#include "common.cuh"
#include "kernels.h"
#include "sink.cuh"
#include "sink_tc.cuh"
#include "tcgen05_heads.cuh"
#include "tma_host.h"

namespace based {
namespace {

using namespace tc;

constexpr int C = 128;                       // rows of a tile
constexpr int kRowWarps = 8;                 // 2 slots x 4 lane quadrants
constexpr int kThreads = 384;                // 4 control warps, one of them idle: whole warpgroups split the registers
// Registers per thread: 168 at launch (384 x 168 of the SM's 65,536); the rows hold a row's weights.
constexpr int kRowRegs = 216, kControlRegs = 72;   // 2 x 216 + 72 = 3 x 168
template <int D>
struct FwdLayout {
    static constexpr uint32_t BLOCK = C * 128;               // 64 columns x 128 rows, 128-byte swizzle
    static constexpr uint32_t TILE = C * D * 2;
    static constexpr int STAGES = D == 128 ? 2 : 4;          // K and V tiles each
    static constexpr uint32_t OFF_Q = 0;                     // two slots
    static constexpr uint32_t OFF_K = OFF_Q + 2 * TILE;
    static constexpr uint32_t OFF_V = OFF_K + STAGES * TILE;
    static constexpr uint32_t OFF_BAR = OFF_V + STAGES * TILE;
    static constexpr uint32_t SMEM_BYTES = OFF_BAR + 512 + 1024;   // + alignment slack
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
    static constexpr uint32_t COL_S = 0, COL_O = 256;        // slot s at + 128 s, + D s
};

enum {
    FB_QF = 0,                // [2] TMA: Q of the slot landed
    FB_QE = 2,                // [2] MMA commit: Q of the slot no longer read
    FB_SF = 4,                // [2] MMA commit: S of the slot ready (and O at rest)
    FB_PF = 6,                // [2] row warps: P of the slot written
    FB_OF = 8,                // [2] MMA commit: O of the slot complete
    FB_OE = 10,               // [2] row warps: O of the slot read out
    FB_KF = 12,               // [4] TMA: K of stage s landed
    FB_KE = 16,               // [4] both slots' MMA commits: K of stage s read
    FB_VF = 20,               // [4]
    FB_VE = 24,               // [4]
    FB_T = 28,                // [2] row warps: the slot has formed a step's weights (its turn is over)
    FB_NUM = 30
};

struct FwdParams {
    const int64_t* lengths;
    View q, k, v, y;
    float* lse;
    unsigned* status;
    int B, Hq, Hkv, N, w, n_sink, sk;        // sk: n_sink rounded up to 16
    FastDiv by_x, by_h, by_group;            // units per tile row; slots' heads per sequence; heads per key/value head
    int nt, pair_heads, units, wide_y;       // wide_y: 32-byte rows
    float c, scale;                          // c: scale * log2(e)
    unsigned debug;
    int fill;                                // the cache's fill follows
};

struct FwdCtx {
    uint32_t sbase;
    uint64_t* bars;
    volatile int* abort_flag;
    volatile int* redo;                      // some row came out non-finite
    unsigned* status;
};

__device__ __forceinline__ bool fwait(const FwdCtx& cx, int bar, uint32_t parity) {
    return mbar_wait(&cx.bars[bar], parity, cx.abort_flag, cx.status);
}

__device__ __forceinline__ bool fwait_joint(const FwdCtx& cx, int bar, uint32_t parity) {
    return mbar_wait_joint(&cx.bars[bar], parity, cx.abort_flag, cx.status);
}

// After an abort: wait (bounded) for this thread's own last asynchronous work.
__device__ __forceinline__ void fdrain(const FwdCtx& cx, int bar, uint32_t parity) {
    if (!*cx.abort_flag || bar < 0) return;
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait(&cx.bars[bar], parity) && global_ns() - t0 < kWaitLimitNs) {}
}

// Unit u: its two slots and the steps both roles walk. Long sweeps (late tiles)
// first, and blocks that run together share their key/value tiles in L2.
struct FwdUnit {
    int b, hk, len;
    int head[2], tile[2], lo[2];
    bool on[2], sink[2];                     // slot has rows to compute; needs the sink block
    int lo_all, hi_all, sink_step, steps;

    __device__ __forceinline__ FwdUnit(const FwdParams& p, int u, unsigned* status) {
        const int row = p.by_x.div(u), x = u - row * (int)p.by_x.d;
        b = p.by_h.div(x);
        const int hx = x - b * (int)p.by_h.d;
        if (p.pair_heads) {
            head[0] = 2 * hx;
            head[1] = head[0] + 1;
            tile[0] = tile[1] = p.nt - 1 - row;
        } else {
            head[0] = head[1] = hx;
            tile[0] = 2 * ((p.nt + 1) / 2 - 1 - row);
            tile[1] = tile[0] + 1;
        }
        hk = p.by_group.div(head[0]);
        len = p.N;
        if (p.lengths != nullptr) {
            const int64_t n = p.lengths[b];
            if ((n < 0 || n > p.N) && status != nullptr) atomicOr(status, DEV_ERR_RANGE);
            len = n < 0 ? 0 : n > p.N ? p.N : (int)n;
        }
        lo_all = 0x7fffffff;
        hi_all = -1;
        sink_step = 0;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            on[s] = tile[s] * C < len;
            lo[s] = max(0, tile[s] * C - p.w + 1) / C;
            sink[s] = on[s] && p.n_sink > 0 && lo[s] > 0;
            if (on[s]) {
                lo_all = min(lo_all, lo[s]);
                hi_all = max(hi_all, tile[s]);
            }
            sink_step |= sink[s] ? 1 : 0;
        }
        steps = hi_all < 0 ? 0 : hi_all - lo_all + 1 + sink_step;
    }
    __device__ __forceinline__ bool is_sink(int j) const { return j < sink_step; }
    __device__ __forceinline__ int key_tile(int j) const { return lo_all + j - sink_step; }
    __device__ __forceinline__ int first(int s) const { return sink[s] ? 0 : lo[s] - lo_all + sink_step; }
};

// One slot of a unit (s selects, so that nothing is indexed in memory).
struct FwdSlot {
    int head, tile, lo, first, last;
    bool on, sink;
    __device__ __forceinline__ FwdSlot(const FwdUnit& u, int s) {
        head = s ? u.head[1] : u.head[0];
        tile = s ? u.tile[1] : u.tile[0];
        lo = s ? u.lo[1] : u.lo[0];
        on = s ? u.on[1] : u.on[0];
        sink = s ? u.sink[1] : u.sink[0];
        first = sink ? 0 : lo - u.lo_all + u.sink_step;
        last = tile - u.lo_all + u.sink_step;
    }
    __device__ __forceinline__ int count() const { return on ? tile - lo + 1 + (sink ? 1 : 0) : 0; }
    __device__ __forceinline__ bool active(const FwdUnit& u, int j) const {
        return on && (j < u.sink_step ? sink : j >= lo - u.lo_all + u.sink_step && j <= last);
    }
};

// ------------------------------------------------------------------ TMA loads (warp 8, lane 0)
template <int D>
__device__ __forceinline__ void fwd_load(const FwdCtx& cx, const FwdParams& p, const CUtensorMap* mq,
                                         const CUtensorMap* mk, const CUtensorMap* mv, const CUtensorMap* mks,
                                         const CUtensorMap* mvs) {
    using L = FwdLayout<D>;
    int gs = 0, nq[2] = {0, 0}, last = -1;
    uint32_t lastp = 0;
    for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
        const FwdUnit un(p, u, p.status);
        // Q of a slot goes in just before the step that reads it first, so that the
        // wait for its buffer does not hold back the other slot's keys.
        for (int j = 0; j < un.steps; ++j, ++gs) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (!un.on[s] || un.first(s) != j) continue;
                if (nq[s] > 0 && !fwait(cx, FB_QE + s, (nq[s] - 1) & 1)) { fdrain(cx, last, lastp); return; }
                mbar_expect_tx(&cx.bars[FB_QF + s], L::TILE);
#pragma unroll
                for (int h = 0; h < D / 64; ++h)
                    tma_load_4d(cx.sbase + L::OFF_Q + s * L::TILE + h * L::BLOCK, mq, &cx.bars[FB_QF + s], 64 * h,
                                un.tile[s] * C, un.head[s], un.b);
                last = FB_QF + s;
                lastp = nq[s]++ & 1;
            }
            const int st = gs % L::STAGES;
            const uint32_t ph = (gs / L::STAGES) & 1;
            const bool sink = un.is_sink(j);
            const uint32_t blk = sink ? p.sk * 128u : L::BLOCK;
            const int row = sink ? 0 : un.key_tile(j) * C;
            if (gs >= L::STAGES && !fwait(cx, FB_KE + st, ph ^ 1)) { fdrain(cx, last, lastp); return; }
            mbar_expect_tx(&cx.bars[FB_KF + st], blk * (D / 64));
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
                tma_load_4d(cx.sbase + L::OFF_K + st * L::TILE + h * blk, sink ? mks : mk, &cx.bars[FB_KF + st], 64 * h,
                            row, un.hk, un.b);
            last = FB_KF + st, lastp = ph;
            if (gs >= L::STAGES && !fwait(cx, FB_VE + st, ph ^ 1)) { fdrain(cx, last, lastp); return; }
            mbar_expect_tx(&cx.bars[FB_VF + st], blk * (D / 64));
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
                tma_load_4d(cx.sbase + L::OFF_V + st * L::TILE + h * blk, sink ? mvs : mv, &cx.bars[FB_VF + st], 64 * h,
                            row, un.hk, un.b);
            last = FB_VF + st, lastp = ph;
        }
    }
    fdrain(cx, last, lastp);
}

// ------------------------------------------------------------------ MMAs (warps 9, 10: slots 0, 1)
template <int D>
__device__ __forceinline__ void fwd_mma(const FwdCtx& cx, const FwdParams& p, uint32_t tmem, int s) {
    using L = FwdLayout<D>;
    const auto wait = [&](int bar, uint32_t parity) {
        return mbar_wait_warp(&cx.bars[bar], parity, cx.abort_flag, cx.status);
    };
    int gs = 0;                              // ring step
    int nq = 0, np = 0;                      // units and weight tiles of the slot so far
    const uint32_t id_s_sink = idesc_bf16_f32(C, p.sk, false, false);
    constexpr uint32_t id_s = idesc_bf16_f32(C, C, false, false), id_o = idesc_bf16_f32(C, D, false, true);
    // Descriptors of the first stage; tiles and K steps add to their address field (16-byte units).
    const uint64_t dq = smem_desc_sw128(cx.sbase + L::OFF_Q + s * L::TILE, 16, 1024),
                   dk = smem_desc_sw128(cx.sbase + L::OFF_K, 16, 1024),
                   dv = smem_desc_sw128(cx.sbase + L::OFF_V, L::BLOCK, 1024),
                   dv_sink = smem_desc_sw128(cx.sbase + L::OFF_V, p.sk * 128u, 1024);
    const uint32_t to = tmem + L::COL_O + D * s, ts = tmem + L::COL_S + 128 * s;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
        const FwdUnit un(p, u, nullptr);
        const FwdSlot sl(un, s);
        // S = Q K^T of ring step g, O += P V of ring step g.
        const auto scores = [&](int g, bool sink, bool first, bool final) {
            const int st = g % L::STAGES;
            ok = wait(FB_KF + st, (g / L::STAGES) & 1);
            if (ok && first) ok = wait(FB_QF + s, nq++ & 1);
            if (!ok) return;
            tc_fence_after();
            const uint64_t k0 = dk + st * (L::TILE >> 4);
            if (elect_one()) {
                if (sink) {
                    for (int k = 0; k < D / 16; ++k)
                        mma_bf16(ts, dq + (k >> 2) * (L::BLOCK >> 4) + (k & 3) * 2,
                                 k0 + (k >> 2) * p.sk * 8 + (k & 3) * 2, id_s_sink, k > 0);
                } else {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_bf16(ts, dq + ((k >> 2) * (L::BLOCK >> 4) + (k & 3) * 2),
                                 k0 + ((k >> 2) * (L::BLOCK >> 4) + (k & 3) * 2), id_s, k > 0);
                }
                mma_commit(&cx.bars[FB_SF + s]);
                mma_commit(&cx.bars[FB_KE + st]);
                if (final) mma_commit(&cx.bars[FB_QE + s]);
            }
            __syncwarp();
        };
        const auto product = [&](int g, bool sink, bool first, bool final) {
            const int st = g % L::STAGES;
            ok = wait(FB_VF + st, (g / L::STAGES) & 1);
            if (ok && first && nq > 1) ok = wait(FB_OE + s, (nq - 2) & 1);
            ok = ok && wait(FB_PF + s, np++ & 1);
            if (!ok) return;
            tc_fence_after();
            const uint64_t v = (sink ? dv_sink : dv) + st * (L::TILE >> 4);
            if (elect_one()) {
                if (sink) {
                    for (int k = 0; k < p.sk / 16; ++k)
                        mma_bf16_ts(to, ts + 8 * k, v + k * 128, id_o, (!first || k > 0) ? 1u : 0u);
                } else {
                    mma_bf16_ts(to, ts, v, id_o, first ? 0u : 1u);
#pragma unroll
                    for (int k = 1; k < C / 16; ++k) mma_bf16_ts(to, ts + 8 * k, v + k * 128, id_o, 1u);
                }
                mma_commit(&cx.bars[FB_VE + st]);
                if (final) mma_commit(&cx.bars[FB_OF + s]);
            }
            __syncwarp();
        };
        // A step that the other slot alone uses is released at once.
        const auto skip = [&](int g) {
            ok = wait(FB_KF + g % L::STAGES, (g / L::STAGES) & 1) && wait(FB_VF + g % L::STAGES, (g / L::STAGES) & 1);
            if (!ok) return;
            if (elect_one()) {
                mbar_arrive(&cx.bars[FB_KE + g % L::STAGES]);
                mbar_arrive(&cx.bars[FB_VE + g % L::STAGES]);
            }
            __syncwarp();
        };
        int before = -1;                     // the step whose P V is outstanding
        for (int j = 0; ok && j < un.steps; ++j) {
            if (!sl.active(un, j)) {
                if (before >= 0) product(gs + before, un.is_sink(before), before == sl.first, before == sl.last);
                before = -1;
                if (ok) skip(gs + j);
                continue;
            }
            if (before >= 0) product(gs + before, un.is_sink(before), before == sl.first, before == sl.last);
            if (ok) scores(gs + j, un.is_sink(j), j == sl.first, j == sl.last);
            before = j;
        }
        if (ok && before >= 0) product(gs + before, un.is_sink(before), before == sl.first, before == sl.last);
        gs += un.steps;
    }
    // Every MMA of this slot has completed: O of the last unit is the last commit.
    if (ok && nq > 0) wait(FB_OF + s, (nq - 1) & 1);
    if (nq > 0) fdrain(cx, FB_OF + s, (nq - 1) & 1);
}

// ------------------------------------------------------------------ rows (warps 0-3, 4-7)

// Thread = row r of slot s = TMEM lane r.
template <int D>
__device__ __forceinline__ void fwd_rows(const FwdCtx& cx, const FwdParams& p, uint32_t tmem, int s, int wq, int lane) {
    using L = FwdLayout<D>;
    const int r = wq * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t ts = tl + L::COL_S + 128 * s, to = tl + L::COL_O + D * s;
    int gs = 0, np = 0, nq = 0, nt = 0;                      // ring steps, weight tiles, units, turns so far
    for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
        int paired;                                          // steps on which the slots take turns
        int lo, tile, len, g0;                               // the slot's key tiles lo .. tile; ring step of tile 0
        const int gu = gs;                                   // the unit's first ring step: the sink block, if any
        bool on, sinks;
        {
            const FwdUnit un(p, u, nullptr);
            const FwdSlot sl(un, s);
            on = sl.on, sinks = sl.sink, lo = sl.lo, tile = sl.tile, len = un.len;
            g0 = gs + un.sink_step - un.lo_all;
            gs += un.steps;
            const FwdSlot other(un, s ^ 1);
            paired = min(sl.count(), other.count());
        }
        const int i0 = tile * C, i = i0 + r;
        float m = -INFINITY, l0 = 0.f, l1 = 0.f;             // m: of the scores times c
        bool first = true;
        for (int t = sinks ? -1 : lo; on && t <= tile; t = t < 0 ? lo : t + 1) {   // -1: the sink block
            const bool sink = t < 0;
            const int j0 = sink ? 0 : t * C;
            // Visible columns, 32 per word: [cl, ch) are inside the window, and the sinks of
            // tile 0 stay visible below it.
            uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u};
            const bool edge = sink || j0 + C > i0 || j0 < i0 + C - p.w;
            uint32_t any = 15u;                              // words some row of the warp sees
            if (edge) {
                const int ch = sink ? p.n_sink : i - j0 + 1, cl = sink ? 0 : i - p.w + 1 - j0;
                const int cs = j0 == 0 ? p.n_sink : 0;
                any = 0u;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    vis[q] = low_bits(ch - 32 * q) & (~low_bits(cl - 32 * q) | low_bits(cs - 32 * q));
                    any |= __any_sync(0xffffffffu, vis[q] != 0u) ? 1u << q : 0u;
                }
            }
            if (!fwait_joint(cx, FB_SF + s, np & 1)) return;
            tc_fence_after();
            // The row's new maximum decides whether to rescale, then the weights; those of
            // columns 32 q .. overlay scores that are read already.
            const auto grow = [&](float mt) {
                mt *= p.c;                                   // -inf stays: c > 0
                const bool grown = mt > m + 8.0f;
                if (__any_sync(0xffffffffu, grown)) {
                    const float al = grown ? ex2(m - mt) : 1.0f;   // 0 the first time
                    l0 *= al;
                    l1 *= al;
                    if (grown) m = mt;
                    if (!first) scale_row<D>(to, al);
                }
                return m == -INFINITY ? 0.f : m;
            };
            // The slots take turns at the exponentials, slot 0 first: left alone they fall into
            // step, and then either both form weights or both wait for the tensor core.
            const bool turns = paired > 0;
            --paired;
            const auto take_turn = [&]() { return !turns || (s == 0 && nt == 0) || fwait_joint(cx, FB_T + (s ^ 1), (nt - (s ^ 1)) & 1); };
            if (!edge) {
                float sv[128];
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld32(ts + 32 * q, sv + 32 * q);
                tmem_ld_wait();
                const float mu = grow(fmaxf(fmaxf(max32(sv), max32(sv + 32)), fmaxf(max32(sv + 64), max32(sv + 96))));
                if (!take_turn()) return;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t pb[16];
                    weights32(sv + 32 * q, p.c, mu, pb, l0, l1);
                    tmem_st16(ts + 16 * q, pb);
                }
            } else {
                // A tile at the window's edge: only the words some row of the warp sees, read
                // twice (the mask and all scores together would not fit in registers).
                float mt = -INFINITY;
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    if (!((any >> q) & 1u)) continue;
                    float sv[32];
                    tmem_ld32(ts + 32 * q, sv);
                    tmem_ld_wait();
                    WordMask(q == 0 ? vis[0] : q == 1 ? vis[1] : q == 2 ? vis[2] : vis[3]).apply(sv, -INFINITY);
                    mt = fmaxf(mt, max32(sv));
                }
                const float mu = grow(mt);
                if (!take_turn()) return;
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    uint32_t pb[16];
                    if ((any >> q) & 1u) {
                        float sv[32];
                        tmem_ld32(ts + 32 * q, sv);
                        tmem_ld_wait();
                        WordMask(q == 0 ? vis[0] : q == 1 ? vis[1] : q == 2 ? vis[2] : vis[3]).apply(sv, -INFINITY);
                        weights32(sv, p.c, mu, pb, l0, l1);
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) pb[e] = 0u;
                    }
                    tmem_st16(ts + 16 * q, pb);
                }
            }
            if (turns) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&cx.bars[FB_T + s]);
                ++nt;
            }
            // Rows of V that no weight may meet: padding in the tile of the sequence's end
            // (the tensor's own end is zero-filled), tokens after the sinks in their block.
            const int v0 = sink ? p.n_sink : len - j0, v1 = sink ? p.sk : min(C, p.N - j0);
            if ((sink || t == tile) && v0 < v1) {
                const int g = sink ? gu : g0 + t, st = g % L::STAGES;
                if (!fwait_joint(cx, FB_VF + st, (g / L::STAGES) & 1)) return;
                if (r >= v0 && r < v1) {
                    const uint32_t blk = sink ? p.sk * 128u : L::BLOCK;
                    const uint32_t row = cx.sbase + L::OFF_V + st * L::TILE + r * 128;
#pragma unroll
                    for (int h = 0; h < D / 64; ++h)
#pragma unroll
                        for (int q = 0; q < 8; ++q) st_shared_v4(row + h * blk + 16 * q, make_uint4(0, 0, 0, 0));
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&cx.bars[FB_PF + s]);
            ++np;
            first = false;
        }
        if (tile >= p.nt) continue;                          // the odd tile's partner: nothing there
        const FwdUnit un(p, u, nullptr);
        const int head = s ? un.head[1] : un.head[0];
        // ---- the slot's outputs
        const bool live = on && i < len;
        const float l = l0 + l1;
        const float inv = live ? 1.0f / l : 0.f;
        if (p.lse != nullptr && i < p.N)
            p.lse[((size_t)un.b * p.Hq + head) * p.N + i] = live ? m * kLn2 + logf(l) : -INFINITY;
        if (on) {
            if (!fwait_joint(cx, FB_OF + s, nq & 1)) return;
            tc_fence_after();
        }
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y.p) + un.b * p.y.sb + head * p.y.sh + i * p.y.sn;
        float odd = 0.f;                                     // NaN where an output is not finite
#pragma unroll
        for (int h = 0; h < D / 32; ++h) {
            float o[32];
            if (on) {
                tmem_ld32(to + 32 * h, o);
                tmem_ld_wait();
                if (h == D / 32 - 1) {                       // O may be overwritten
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&cx.bars[FB_OE + s]);
                }
            }
            if (i < p.N) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float x[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        x[e] = live ? o[16 * q + e] * inv : 0.f;
                        odd = fmaf(x[e], 0.f, odd);
                    }
                    store16(y + 32 * h + 16 * q, pack_bf16x8(x), pack_bf16x8(x + 8), p.wide_y);
                }
            }
            __syncwarp();
        }
        if (live && odd != 0.f) *cx.redo = 1;
        __syncwarp();
        if (on) ++nq;
    }
}

// Non-finite rows of the block's units, again from their definition.
template <int D>
__device__ __noinline__ void fwd_redo(const FwdParams& p, int warp) {
    for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
        const FwdUnit un(p, u, nullptr);
#pragma unroll
        for (int s = 0; s < 2; ++s)
            redo_rows<__nv_bfloat16, D>(p, un.b, un.head[s], un.hk, un.tile[s] * C, C, un.len, un.lo[s] * C, 0, warp, kRowWarps);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
sink_fwd_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mks,
                   const __grid_constant__ CUtensorMap mvs, const __grid_constant__ FwdParams p) {
    using L = FwdLayout<D>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    unsigned char* smem = smem_raw + (sbase - raw);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_BAR + 8 * FB_NUM);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_BAR + 8 * FB_NUM + 4);
    const FwdCtx cx{sbase, bars, abort_flag, abort_flag + 1, p.status};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int b = 0; b < FB_NUM; ++b) {
            uint32_t count = 1;
            if (b == FB_PF || b == FB_PF + 1 || b == FB_OE || b == FB_OE + 1 || b == FB_T || b == FB_T + 1)
                count = 4;                                   // warps of a slot
            if ((b >= FB_KE && b < FB_KE + 4) || (b >= FB_VE && b < FB_VE + 4)) count = 2;   // slots
            mbar_init(&bars[b], count);
        }
        *abort_flag = 0;
        *cx.redo = 0;
        mbar_fence_init();
    }
    if (warp == kRowWarps + 1) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();                                  // inputs may come from earlier kernels
    if (p.fill) grid_launch_dependents();                    // the cache's fill may start
    if (warp >= kRowWarps) {
        reg_dec<kControlRegs>();
        if (warp == kRowWarps) {
            if (lane == 0) fwd_load<D>(cx, p, &mq, &mk, &mv, &mks, &mvs);
        } else if (warp <= kRowWarps + 2) {
            if (!(p.debug & DEBUG_SKIP_MMA)) fwd_mma<D>(cx, p, tmem, warp - kRowWarps - 1);
        }
    } else {
        reg_inc<kRowRegs>();
        fwd_rows<D>(cx, p, tmem, warp >> 2, warp & 3, lane);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kRowWarps + 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    // The row warps alone: the others have given their registers away.
    if (*cx.redo && !*abort_flag && warp < kRowWarps) fwd_redo<D>(p, warp);
}

template <int D>
cudaError_t run(const SinkArgs& a, int num_sms, cudaStream_t stream) {
    using L = FwdLayout<D>;
    FwdParams p{};
    p.lengths = a.lengths, p.q = a.q, p.k = a.k, p.v = a.v, p.y = a.y, p.lse = a.lse, p.status = a.status, p.debug = a.debug, p.fill = a.fill;
    p.B = a.B, p.Hq = a.Hq, p.Hkv = a.Hkv, p.N = a.N, p.w = a.w, p.n_sink = a.n_sink;
    p.sk = std::max(16, (a.n_sink + 15) / 16 * 16);
    p.nt = (a.N + C - 1) / C;
    p.pair_heads = (a.Hq / a.Hkv) % 2 == 0;
    p.units = p.pair_heads ? p.nt * a.B * (a.Hq / 2) : (p.nt + 1) / 2 * a.B * a.Hq;
    p.by_x = FastDiv(p.pair_heads ? a.B * (a.Hq / 2) : a.B * a.Hq), p.by_h = FastDiv(p.pair_heads ? a.Hq / 2 : a.Hq);
    p.by_group = FastDiv(a.Hq / a.Hkv);
    p.wide_y = rows_aligned32(a.y);
    // A scale of 0 (equal weights) becomes the least number, so that -inf times it stays -inf
    // and any finite score times it is next to 0.
    p.c = std::max(a.scale * kLog2e, std::numeric_limits<float>::denorm_min());
    p.scale = a.scale;
    CUtensorMap mq, mk, mv, mks, mvs;
    if (!heads_map(&mq, a.q, a, a.Hq, C) || !heads_map(&mk, a.k, a, a.Hkv, C) || !heads_map(&mv, a.v, a, a.Hkv, C) ||
        !heads_map(&mks, a.k, a, a.Hkv, p.sk) || !heads_map(&mvs, a.v, a, a.Hkv, p.sk))
        return cudaErrorInvalidValue;
    auto kern = sink_fwd_tc_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(std::min(p.units, num_sms)), dim3(kThreads), L::SMEM_BYTES, stream, mq, mk, mv, mks,
                      mvs, p);
}

}  // namespace

cudaError_t launch_sink_prefill_tc(const SinkArgs& a, int num_sms, cudaStream_t stream) {
    // Few steps per tile: several small blocks on an SM hide what this pipeline waits for. What
    // counts is the keys a tile sees, at most N, so the crossing moves with N, and whether there
    // are tiles for several blocks. Narrow : wide, us, by batch x tokens and w, 16 heads (4:
    // key/value heads), 4 sinks:
    //   d = 64    16 x 512 all 36 : 39   16 (4) x 700 all 50 : 60   16 x 1024 512 82 : 95, all 107 : 99
    //             8 x 2048 1024 129 : 139, 1536 174 : 156   4 x 4096 2048 211 : 218, all 298 : 273
    //             2 (4) x 8192 3000 300 : 317, 4096 376 : 373   1 (4) x 16384 4096 412 : 431
    //             512 tiles (8 heads x 8192) 2048 72 : 78, 4096 128 : 121   256 tiles (4 x 8192) 512
    //             20 : 21, 1024 30 : 28, 2048 50 : 43   128 tiles (1 x 16384) 512 17 : 20, 1536 35 : 34
    //   d = 128   32 x 128 all 20 : 25   32 x 256 all 43 : 41   4 (4) x 4096 128 82 : 84, 192 91 : 100,
    //             256 101 : 101, 384 120 : 115   2 (4) x 16384 192 177 : 189, 256 197 : 192
    const int w = std::min(a.w, a.N);
    const bool many = (long long)a.B * a.Hq * ((a.N + C - 1) / C) >= 3LL * num_sms;
    if (w <= (a.d == 128 ? 192 : many ? std::max(768, a.N / 2 + 256) : 768)) return launch_sink_prefill_narrow(a, num_sms, stream);
    return a.d == 64 ? run<64>(a, num_sms, stream) : run<128>(a, num_sms, stream);
}

}  // namespace based
