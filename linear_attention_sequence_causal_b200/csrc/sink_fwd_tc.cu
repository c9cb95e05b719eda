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
// TMEM lane), warp 8 the TMA loads, warp 9 TMEM allocation and all MMAs.
// TMEM: S0, S1 (128 columns each, P over the first 64), O0, O1 (d columns each).
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "sink.cuh"
#include "tcgen05.cuh"
#include "tma_host.h"

namespace based {
namespace {

using namespace tc;

constexpr int C = 128;                       // rows of a tile
constexpr int kThreads = 384;                // three warpgroups, for the register split
// Registers per thread: 168 at launch (384 x 168); the rows hold a whole score row.
constexpr int kRowRegs = 232, kControlRegs = 40;   // 2 x 232 + 40 = 3 x 168
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

template <int D>
struct FwdLayout {
    static constexpr uint32_t BLOCK = C * 128;               // 64 columns x 128 rows, 128-byte swizzle
    static constexpr uint32_t TILE = C * D * 2;
    static constexpr int STAGES = D == 128 ? 2 : 4;          // K and V tiles each
    static constexpr uint32_t OFF_Q = 0;                     // two slots
    static constexpr uint32_t OFF_K = OFF_Q + 2 * TILE;
    static constexpr uint32_t OFF_V = OFF_K + STAGES * TILE;
    static constexpr uint32_t OFF_Y = OFF_V + STAGES * TILE; // 64 output columns per slot, on their way out
    static constexpr uint32_t OFF_BAR = OFF_Y + 2 * BLOCK;
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
    FB_YF = 12,               // [2] row threads: staged output columns written
    FB_YE = 14,               // [2] the store's thread: staged columns read by TMA
    FB_KF = 16,               // [4] TMA: K of stage s landed
    FB_KE = 20,               // [4] MMA commit: K of stage s read
    FB_VF = 24,               // [4]
    FB_VE = 28,               // [4]
    FB_NUM = 32
};

struct FwdParams {
    const int64_t* lengths;
    float* lse;
    unsigned* status;
    int B, Hq, Hkv, N, w, n_sink, sk;        // sk: n_sink rounded up to 16
    int nt, pair_heads, units;
    float c;                                 // scale * log2(e)
    unsigned debug;
};

struct FwdCtx {
    uint32_t sbase;
    uint64_t* bars;
    volatile int* abort_flag;
    unsigned* status;
};

__device__ __forceinline__ bool fwait(const FwdCtx& cx, int bar, uint32_t parity) {
    return mbar_wait(&cx.bars[bar], parity, cx.abort_flag, cx.status);
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
        if (p.pair_heads) {
            const int hp = p.B * p.Hq / 2;
            const int t = p.nt - 1 - u / hp, x = u % hp;
            b = x / (p.Hq / 2);
            head[0] = 2 * (x % (p.Hq / 2));
            head[1] = head[0] + 1;
            tile[0] = tile[1] = t;
        } else {
            const int bh = p.B * p.Hq, np = (p.nt + 1) / 2;
            const int t = np - 1 - u / bh, x = u % bh;
            b = x / p.Hq;
            head[0] = head[1] = x % p.Hq;
            tile[0] = 2 * t;
            tile[1] = 2 * t + 1;
        }
        hk = head[0] / (p.Hq / p.Hkv);
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
    __device__ __forceinline__ bool active(int s, int j) const {
        if (j < sink_step) return sink[s];
        const int t = lo_all + j - sink_step;
        return on[s] && t >= lo[s] && t <= tile[s];
    }
    __device__ __forceinline__ int first(int s) const { return sink[s] ? 0 : lo[s] - lo_all + sink_step; }
    __device__ __forceinline__ int last(int s) const { return tile[s] - lo_all + sink_step; }
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

// ------------------------------------------------------------------ MMAs (warp 9, lane 0)
template <int D>
__device__ __forceinline__ void fwd_mma(const FwdCtx& cx, const FwdParams& p, uint32_t tmem) {
    using L = FwdLayout<D>;
    int g0 = 0;                              // ring steps of the units before
    int nq[2] = {0, 0};                      // units of the slot so far
    int np[2] = {0, 0};                      // weight tiles of the slot so far
    int last = -1;
    uint32_t lastp = 0;
    const uint32_t id_s_sink = idesc_bf16_f32(C, p.sk, false, false);
    constexpr uint32_t id_s = idesc_bf16_f32(C, C, false, false), id_o = idesc_bf16_f32(C, D, false, true);
    for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
        const FwdUnit un(p, u, nullptr);
        for (int j = 0; j <= un.steps; ++j) {
            const int stk = (g0 + j) % L::STAGES, stv = (g0 + j - 1) % L::STAGES;
            const uint32_t phk = ((g0 + j) / L::STAGES) & 1, phv = ((g0 + j - 1) / L::STAGES) & 1;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (j > 0 && un.active(s, j - 1)) {          // O += P V of step j - 1
                    const bool first = un.first(s) == j - 1;
                    bool ok = fwait(cx, FB_VF + stv, phv) && fwait(cx, FB_PF + s, np[s] & 1);
                    if (ok && first && nq[s] > 1) ok = fwait(cx, FB_OE + s, (nq[s] - 2) & 1);
                    if (!ok) { fdrain(cx, last, lastp); return; }
                    ++np[s];
                    tc_fence_after();
                    const bool sink = un.is_sink(j - 1);
                    const int ks = sink ? p.sk / 16 : C / 16;
                    const uint32_t blk = sink ? p.sk * 128u : L::BLOCK;
                    const uint32_t v = cx.sbase + L::OFF_V + stv * L::TILE;
                    for (int k = 0; k < ks; ++k)
                        mma_bf16_ts(tmem + L::COL_O + D * s, tmem + L::COL_S + 128 * s + 8 * k,
                                    smem_desc_sw128(v + k * 2048, blk, 1024), id_o, (!first || k > 0) ? 1u : 0u);
                    if (un.last(s) == j - 1) mma_commit(&cx.bars[FB_OF + s]);
                }
                if (j < un.steps && un.active(s, j)) {       // S = Q K^T of step j
                    const bool first = un.first(s) == j;
                    bool ok = fwait(cx, FB_KF + stk, phk);
                    if (ok && first) ok = fwait(cx, FB_QF + s, nq[s]++ & 1);
                    if (!ok) { fdrain(cx, last, lastp); return; }
                    tc_fence_after();
                    const bool sink = un.is_sink(j);
                    const uint32_t blk = sink ? p.sk * 128u : L::BLOCK;
                    const uint32_t q = cx.sbase + L::OFF_Q + s * L::TILE, k0 = cx.sbase + L::OFF_K + stk * L::TILE;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_bf16(tmem + L::COL_S + 128 * s,
                                 smem_desc_sw128(q + (k >> 2) * L::BLOCK + (k & 3) * 32, 16, 1024),
                                 smem_desc_sw128(k0 + (k >> 2) * blk + (k & 3) * 32, 16, 1024),
                                 sink ? id_s_sink : id_s, k > 0);
                    mma_commit(&cx.bars[FB_SF + s]);
                    if (un.last(s) == j) mma_commit(&cx.bars[FB_QE + s]);
                }
            }
            if (j > 0) {
                mma_commit(&cx.bars[FB_VE + stv]);
                last = FB_VE + stv, lastp = phv;
            }
            if (j < un.steps) {
                mma_commit(&cx.bars[FB_KE + stk]);
                last = FB_KE + stk, lastp = phk;
            }
        }
        g0 += un.steps;
    }
    if (last >= 0) fwait(cx, last, lastp);                   // every MMA has completed
    fdrain(cx, last, lastp);
}

// ------------------------------------------------------------------ rows (warps 0-3, 4-7)

// The weights of 32 columns: p = 2^(s c - m), packed to bf16; l0, l1 += the unrounded weights.
__device__ __forceinline__ void weights32(const float* s, float c, float m, uint32_t* out, float& l0, float& l1) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float a = ex2(fmaf(s[2 * i], c, -m)), b = ex2(fmaf(s[2 * i + 1], c, -m));
        add_pair(l0, l1, a, b);
        out[i] = pack_bf16x2(a, b);
    }
}

template <int D>
__device__ __forceinline__ void fwd_rows(const FwdCtx& cx, const FwdParams& p, uint32_t tmem, int s, int wq, int lane,
                                         const CUtensorMap* my) {
    using L = FwdLayout<D>;
    const int r = wq * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t ts = tl + L::COL_S + 128 * s, to = tl + L::COL_O + D * s;
    int gs = 0, np = 0, nq = 0, ny = 0;
    for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
        const FwdUnit un(p, u, nullptr);
        // The slot's own values (s selects, so that nothing is indexed in memory).
        const int tile = s ? un.tile[1] : un.tile[0], head = s ? un.head[1] : un.head[0];
        const int lo = s ? un.lo[1] : un.lo[0];
        const bool on = s ? un.on[1] : un.on[0], sinks = s ? un.sink[1] : un.sink[0];
        const int jfirst = sinks ? 0 : lo - un.lo_all + un.sink_step;
        const int i0 = tile * C, i = i0 + r;
        float m = -INFINITY, l0 = 0.f, l1 = 0.f;             // m: of the scores times c
        for (int j = 0; j < un.steps; ++j, ++gs) {
            const bool sink = un.is_sink(j), first = jfirst == j;
            if (sink ? !sinks : !on || un.key_tile(j) < lo || un.key_tile(j) > tile) continue;
            const int j0 = sink ? 0 : un.key_tile(j) * C;
            if (!fwait(cx, FB_SF + s, np & 1)) return;
            tc_fence_after();
            float sv[128];
            const int ncol = sink ? p.sk : C;
            float mt = -INFINITY;
            if (!sink) {
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld32(ts + 32 * q, sv + 32 * q);
                tmem_ld_wait();
                // Columns [cl, ch) are inside the window; sinks of tile 0 stay visible below it.
                if (j0 + C > i0 || j0 < i0 + C - p.w) {
                    const int ch = i - j0, cl = i - p.w + 1 - j0, cs = j0 == 0 ? p.n_sink : 0;
#pragma unroll
                    for (int q = 0; q < 128; ++q)
                        if (q > ch || (q < cl && q >= cs)) sv[q] = -INFINITY;
                }
                float m0 = sv[0], m1 = sv[1], m2 = sv[2], m3 = sv[3];
#pragma unroll
                for (int q = 4; q < 128; q += 8) {
                    m0 = fmaxf(m0, fmaxf(sv[q], sv[q + 1]));
                    m1 = fmaxf(m1, fmaxf(sv[q + 2], sv[q + 3]));
                    if (q + 4 < 128) {
                        m2 = fmaxf(m2, fmaxf(sv[q + 4], sv[q + 5]));
                        m3 = fmaxf(m3, fmaxf(sv[q + 6], sv[q + 7]));
                    }
                }
                mt = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (16 * q < ncol) tmem_ld16(ts + 16 * q, sv + 16 * q);
                }
                tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < 64; ++q) {
                    if (q >= p.n_sink) sv[q] = -INFINITY;
                    mt = fmaxf(mt, sv[q]);
                }
            }
            mt *= p.c;                                       // -inf stays: c > 0
            if (__any_sync(0xffffffffu, mt > m + 8.0f)) {
                const float mn = fmaxf(m, mt);
                const float al = ex2(m - (mn == -INFINITY ? 0.f : mn));
                l0 *= al;
                l1 *= al;
                m = mn;
                if (!first) {
#pragma unroll
                    for (int q = 0; q < D / 16; ++q) {
                        float o[16];
                        tmem_ld16(to + 16 * q, o);
                        tmem_ld_wait();
                        uint32_t ob[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) ob[e] = __float_as_uint(o[e] * al);
                        tmem_st16(to + 16 * q, ob);
                    }
                }
            }
            const float mu = m == -INFINITY ? 0.f : m;
            if (!sink) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t pb[16];
                    weights32(sv + 32 * q, p.c, mu, pb, l0, l1);
                    tmem_st16(ts + 16 * q, pb);
                }
            } else {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (32 * q < ncol) {
                        uint32_t pb[16];
                        weights32(sv + 32 * q, p.c, mu, pb, l0, l1);
                        tmem_st16(ts + 16 * q, pb);
                    }
                }
            }
            // Rows of V that no weight may meet: padding in the tile of the sequence's end
            // (the tensor's own end is zero-filled), tokens after the sinks in their block.
            const int v0 = sink ? p.n_sink : un.len - j0, v1 = sink ? p.sk : min(C, p.N - j0);
            if (v0 < v1) {
                if (!fwait(cx, FB_VF + gs % L::STAGES, (gs / L::STAGES) & 1)) return;
                if (r >= v0 && r < v1) {
                    const uint32_t blk = sink ? p.sk * 128u : L::BLOCK;
                    const uint32_t row = cx.sbase + L::OFF_V + (gs % L::STAGES) * L::TILE + r * 128;
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
        }
        if (tile >= p.nt) continue;                    // the odd tile's partner: nothing there
        // ---- the slot's outputs, 64 columns at a time through shared memory
        const bool live = on && i < un.len;
        const float l = l0 + l1;
        const float inv = 1.0f / l;
        if (p.lse != nullptr && i < p.N)
            p.lse[((size_t)un.b * p.Hq + head) * p.N + i] = live ? m * kLn2 + logf(l) : -INFINITY;
        if (on) {
            if (!fwait(cx, FB_OF + s, nq & 1)) return;
            tc_fence_after();
        }
        const uint32_t stage = cx.sbase + L::OFF_Y + s * L::BLOCK;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
            float o[64];
            if (on) {
                tmem_ld32(to + 64 * h, o);
                tmem_ld32(to + 64 * h + 32, o + 32);
                tmem_ld_wait();
                if (h == D / 64 - 1) {                       // O may be overwritten
                    tc_fence_before();
                    mbar_arrive(&cx.bars[FB_OE + s]);
                }
            }
            if (ny > 0 && !fwait(cx, FB_YE + s, (ny - 1) & 1)) return;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = live ? o[8 * q + e] * inv : 0.f;
                st_shared_v4(stage + sw128_offset(r, q), pack_bf16x8(x));
            }
            fence_proxy_async_smem();
            mbar_arrive(&cx.bars[FB_YF + s]);
            if (r == 0) {
                if (!fwait(cx, FB_YF + s, ny & 1)) return;
                tma_store_4d(my, stage, 64 * h, i0, head, un.b);
                bulk_commit();
                bulk_wait_read_all();
                mbar_arrive(&cx.bars[FB_YE + s]);
            }
            __syncwarp();
            ++ny;
        }
        if (on) ++nq;
    }
    if (r == 0) bulk_wait_all();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
sink_fwd_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mks,
                   const __grid_constant__ CUtensorMap mvs, const __grid_constant__ CUtensorMap my,
                   const __grid_constant__ FwdParams p) {
    using L = FwdLayout<D>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    unsigned char* smem = smem_raw + (sbase - raw);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_BAR + 8 * FB_NUM);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_BAR + 8 * FB_NUM + 4);
    const FwdCtx cx{sbase, bars, abort_flag, p.status};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int b = 0; b < FB_NUM; ++b) {
            uint32_t count = 1;
            if (b == FB_PF || b == FB_PF + 1) count = 4;
            if (b == FB_OE || b == FB_OE + 1 || b == FB_YF || b == FB_YF + 1) count = 128;
            mbar_init(&bars[b], count);
        }
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == 9) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();                                  // inputs may come from earlier kernels
    if (warp >= 8) reg_dec<kControlRegs>();
    if (warp == 8) {
        if (lane == 0) fwd_load<D>(cx, p, &mq, &mk, &mv, &mks, &mvs);
    } else if (warp == 9) {
        if (lane == 0 && !(p.debug & DEBUG_SKIP_MMA)) fwd_mma<D>(cx, p, tmem);
    } else if (warp < 8) {
        reg_inc<kRowRegs>();
        fwd_rows<D>(cx, p, tmem, warp >> 2, warp & 3, lane, &my);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

bool heads_map(CUtensorMap* m, const View& v, const SinkArgs& a, int H, uint32_t rows) {
    return make_tmap_bf16_heads(m, v.p, a.d, a.N, H, a.B, v.sn, v.sh, v.sb, rows);
}

template <int D>
cudaError_t run(const SinkArgs& a, int num_sms, cudaStream_t stream) {
    using L = FwdLayout<D>;
    FwdParams p{};
    p.lengths = a.lengths, p.lse = a.lse, p.status = a.status, p.debug = a.debug;
    p.B = a.B, p.Hq = a.Hq, p.Hkv = a.Hkv, p.N = a.N, p.w = a.w, p.n_sink = a.n_sink;
    p.sk = std::max(16, (a.n_sink + 15) / 16 * 16);
    p.nt = (a.N + C - 1) / C;
    p.pair_heads = (a.Hq / a.Hkv) % 2 == 0;
    p.units = p.pair_heads ? p.nt * a.B * (a.Hq / 2) : (p.nt + 1) / 2 * a.B * a.Hq;
    // A scale of 0 (equal weights) becomes a tiny one, so that -inf times it stays -inf.
    p.c = std::max(a.scale * kLog2e, 1e-30f);
    CUtensorMap mq, mk, mv, mks, mvs, my;
    if (!heads_map(&mq, a.q, a, a.Hq, C) || !heads_map(&mk, a.k, a, a.Hkv, C) || !heads_map(&mv, a.v, a, a.Hkv, C) ||
        !heads_map(&mks, a.k, a, a.Hkv, p.sk) || !heads_map(&mvs, a.v, a, a.Hkv, p.sk) ||
        !heads_map(&my, a.y, a, a.Hq, C))
        return cudaErrorInvalidValue;
    auto kern = sink_fwd_tc_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(std::min(p.units, num_sms)), dim3(kThreads), L::SMEM_BYTES, stream, mq, mk, mv, mks,
                      mvs, my, p);
}

}  // namespace

cudaError_t launch_sink_prefill_tc(const SinkArgs& a, int num_sms, cudaStream_t stream) {
    return a.d == 64 ? run<64>(a, num_sms, stream) : run<128>(a, num_sms, stream);
}

}  // namespace based
