// Backward of the sliding-window attention with sink tokens on the tensor cores (bf16).
//
//   p_ij = 2^(c s_ij - lse_i log2 e), c = scale log2 e;  delta_i = dy_i . y_i
//   dS_ij = p_ij (dy_i . v_j - delta_i)
//   dq_i = scale sum_j dS_ij k_j, dk_j = scale sum_i dS_ij q_i, dv_j = sum_i p_ij dy_i
//
// Two persistent kernels, each one block per SM. Both form the scores again, so that
// every output row belongs to one block and nothing is added atomically (7 products
// per tile pair instead of 5).
//   DQ   unit = a query tile of a head; steps = the sink block, then its key tiles:
//        S = Q K^T, X = dY V^T, dQ += dS K. It also forms delta and leaves
//        -lse log2 e and delta, padded to whole tiles, in the workspace.
//   DKV  unit = a key tile of a key/value head; steps = (head of the group, query
//        tile): S = K Q^T, X = V dY^T, dV += P dY, dK += dS Q (P, dS transposed: rows
//        are keys). The sinks' pairs outside the window are units of their own, whose
//        fp32 partials a last launch joins (see SinkSplit).
//
// P and dS overlay the S and X they come from, so the accumulators fit beside them.
// The rows work in two phases, weights (which need S) and dS (which needs X), and the
// tensor core runs one phase's products during the other: DKV issues dV(n), S(n + 1)
// once the weights of step n stand, dK(n), X(n + 1) once its dS stand; DQ has two S
// buffers and issues S(n + 1) ahead, then dQ(n), X(n + 1).
//
// Roles (640 threads): warps 0-15 the rows (thread = TMEM lane x 32 columns), warp 16
// the TMA loads, warp 17 TMEM allocation and the MMAs (18, 19 idle).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "sink.cuh"
#include "sink_tc.cuh"
#include "tcgen05.cuh"
#include "tma_host.h"

namespace based {
namespace {

using namespace tc;

constexpr int C = 128;
constexpr int kRowWarps = 16;
constexpr int kThreads = 640;

template <int D, bool DKV>
struct BwdLayout {
    static constexpr uint32_t BLOCK = C * 128;               // 64 columns x 128 rows, 128-byte swizzle
    static constexpr uint32_t TILE = C * D * 2;
    static constexpr int OWN = D == 64 ? 2 : 1;              // buffers of the unit's own two tiles
    static constexpr int STAGES = D == 64 ? 4 : 2;           // ring stages of the other side's two tiles
    static constexpr uint32_t OFF_OWN = 0;                   // [OWN][2 tiles]: Q, dY (DQ) or K, V (DKV)
    static constexpr uint32_t OFF_A = OFF_OWN + OWN * 2 * TILE;       // [STAGES]: K (DQ) or Q (DKV)
    static constexpr uint32_t OFF_B = OFF_A + STAGES * TILE;          // [STAGES]: V (DQ) or dY (DKV)
    static constexpr uint32_t OFF_ROW = OFF_B + STAGES * TILE;        // DKV [STAGES][2][128]: -lse log2 e, delta
    static constexpr uint32_t OFF_RED = OFF_ROW + STAGES * 2 * C * 4; // DQ [2][4][128]: partial delta
    static constexpr uint32_t OFF_BAR = OFF_RED + 2 * 4 * C * 4;
    static constexpr uint32_t SMEM_BYTES = OFF_BAR + 512 + 1024;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
    // DKV: S, X, dV, dK. DQ: two S, X, dQ.
    static constexpr uint32_t COL_S = 0, COL_X = DKV ? 128 : 256;
    static constexpr uint32_t COL_ACC = DKV ? 256 : 384;     // DKV: dV, then dK at + D
};

enum {
    GB_OWNF = 0,              // [2] TMA: own tiles landed
    GB_OWNE = 2,              // [2] MMA commit: own tiles no longer read
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
    GB_RED,                   // DQ row warps: partial deltas written
    GB_NUM
};

struct BwdParams {
    const int64_t* lengths;
    const float* lse;
    View y, dy, dq, dk, dv;
    float* nl2;                              // [B Hq][npad]: -lse log2 e
    float* delta;                            // [B Hq][npad]
    float* partial;
    unsigned* status;
    SinkSplit sp;
    int B, Hq, Hkv, N, w, n_sink, sk, nt, npad, units;
    float c, scale;
    unsigned debug;
};

struct BwdCtx {
    uint32_t sbase;
    uint64_t* bars;
    volatile int* abort_flag;
    unsigned* status;
};

__device__ __forceinline__ bool gwait(const BwdCtx& cx, int bar, uint32_t parity) {
    return mbar_wait(&cx.bars[bar], parity, cx.abort_flag, cx.status);
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

__device__ __forceinline__ int bwd_len(const BwdParams& p, int b) {
    if (p.lengths == nullptr) return p.N;
    const int64_t n = p.lengths[b];
    return n < 0 ? 0 : n > p.N ? p.N : (int)n;
}

// A walk over the units of a block and their steps; both kernels' roles take the same
// walk. Steps: DQ the sink block (t = -1), then key tiles lo .. tile; DKV the pairs
// (head, query tile) of the unit's stretch, without tiles of padding.
struct DqWalk {
    int u, b, h, hk, tile, lo, len;
    int t;                                   // the current step's key tile, -1: the sink block
    bool some;                               // the unit has steps

    __device__ __forceinline__ void start(const BwdParams& p, int unit) {
        u = unit;
        if (u >= p.units) return;
        const int bh = p.B * p.Hq;
        tile = p.nt - 1 - u / bh;            // long sweeps first
        b = (u % bh) / p.Hq;
        h = (u % bh) % p.Hq;
        hk = h / (p.Hq / p.Hkv);
        len = bwd_len(p, b);
        lo = max(0, tile * C - p.w + 1) / C;
        some = tile * C < len;
        t = p.n_sink > 0 && lo > 0 ? -1 : lo;
    }
    __device__ __forceinline__ bool last() const { return t == tile; }
    __device__ __forceinline__ void next() { t = t < 0 ? lo : t + 1; }
};

struct KvWalk {
    int u, b, hk, kt, chunk, len;
    int h, t;                                // the current step: query head and tile
    int t0, tv, left, span;                  // tiles t0 .. tv - 1 are real; list entries left (this one too)
    bool some;

    __device__ __forceinline__ void start(const BwdParams& p, int unit) {
        u = unit;
        if (u >= p.units) return;
        const SinkUnit x = sink_unit(p.sp, u, p.B, p.Hkv);
        b = x.b, hk = x.hk, kt = x.kt, chunk = x.chunk;
        len = bwd_len(p, b);
        t0 = x.t0;
        span = x.span;
        tv = min(x.t0 + x.span, (len + C - 1) / C);
        h = hk * p.sp.group + x.s0 / x.span;
        t = x.t0 + x.s0 % x.span;
        left = x.s1 - x.s0;
        if (t >= tv) skip();
        some = tv > t0 && kt * C < len && left > 0;
    }
    __device__ __forceinline__ void skip() {                 // to the next head's first tile
        left -= t0 + span - t;
        t = t0;
        ++h;
    }
    // Entries after this one: in this head, or (with at least one real tile) in a later one.
    __device__ __forceinline__ bool last() const { return t + 1 < tv ? left <= 1 : left - (t0 + span - t) <= 0; }
    __device__ __forceinline__ void next() {
        if (t + 1 < tv) {
            ++t;
            --left;
        } else {
            skip();
        }
    }
};

// ------------------------------------------------------------------ TMA loads (warp 16, lane 0)
struct BwdMaps {
    const CUtensorMap *own0, *own1, *a, *b, *a_sink, *b_sink;
};

template <int D, bool DKV, typename Walk>
__device__ __forceinline__ void bwd_load(const BwdCtx& cx, const BwdParams& p, const BwdMaps& m) {
    using L = BwdLayout<D, DKV>;
    int g = 0, nu = 0, last = -1;
    uint32_t lastp = 0;
    Walk wk;
    for (wk.start(p, blockIdx.x); wk.u < p.units; wk.start(p, wk.u + gridDim.x)) {
        if (!wk.some) continue;
        const int ob = nu % L::OWN;
        if (nu >= L::OWN && !gwait(cx, GB_OWNE + ob, (nu / L::OWN - 1) & 1)) { gdrain(cx, last, lastp); return; }
        int own_row, own_head;
        if constexpr (DKV) own_row = wk.kt * C, own_head = wk.hk;
        else own_row = wk.tile * C, own_head = wk.h;
        mbar_expect_tx(&cx.bars[GB_OWNF + ob], 2 * L::TILE);
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
            const uint32_t o = cx.sbase + L::OFF_OWN + ob * 2 * L::TILE + h * L::BLOCK;
            tma_load_4d(o, m.own0, &cx.bars[GB_OWNF + ob], 64 * h, own_row, own_head, wk.b);
            tma_load_4d(o + L::TILE, m.own1, &cx.bars[GB_OWNF + ob], 64 * h, own_row, own_head, wk.b);
        }
        last = GB_OWNF + ob, lastp = (nu / L::OWN) & 1;
        ++nu;
        for (;;) {
            const int st = g % L::STAGES;
            const uint32_t ph = (g / L::STAGES) & 1;
            uint32_t blk = L::BLOCK;
            int row, head;
            bool sink = false;
            if constexpr (DKV) {
                row = wk.t * C, head = wk.h;
            } else {
                sink = wk.t < 0;
                row = sink ? 0 : wk.t * C, head = wk.hk;
                if (sink) blk = p.sk * 128u;
            }
            const size_t vec = DKV ? ((size_t)wk.b * p.Hq + head) * p.npad + row : 0;
            const uint32_t rows = cx.sbase + L::OFF_ROW + st * 2 * C * 4;
            if (g >= L::STAGES && !gwait(cx, GB_AE + st, ph ^ 1)) { gdrain(cx, last, lastp); return; }
            mbar_expect_tx(&cx.bars[GB_AF + st], blk * (D / 64) + (DKV ? 2 * C * 4 : 0));
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
                tma_load_4d(cx.sbase + L::OFF_A + st * L::TILE + h * blk, sink ? m.a_sink : m.a, &cx.bars[GB_AF + st],
                            64 * h, row, head, wk.b);
            if constexpr (DKV) {                             // with Q: released with it, after the last rows read them
                bulk_load(rows, p.nl2 + vec, C * 4, &cx.bars[GB_AF + st]);
                bulk_load(rows + C * 4, p.delta + vec, C * 4, &cx.bars[GB_AF + st]);
            }
            last = GB_AF + st, lastp = ph;
            if (g >= L::STAGES && !gwait(cx, GB_BE + st, ph ^ 1)) { gdrain(cx, last, lastp); return; }
            mbar_expect_tx(&cx.bars[GB_BF + st], blk * (D / 64));
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
                tma_load_4d(cx.sbase + L::OFF_B + st * L::TILE + h * blk, sink ? m.b_sink : m.b, &cx.bars[GB_BF + st],
                            64 * h, row, head, wk.b);
            last = GB_BF + st, lastp = ph;
            ++g;
            if (wk.last()) break;
            wk.next();
        }
    }
    gdrain(cx, last, lastp);
}

// ------------------------------------------------------------------ MMAs (warp 17)
template <int D, bool DKV, typename Walk>
__device__ __forceinline__ void bwd_mma(const BwdCtx& cx, const BwdParams& p, uint32_t tmem) {
    using L = BwdLayout<D, DKV>;
    constexpr uint32_t id_s = idesc_bf16_f32(C, C, false, false), id_acc = idesc_bf16_f32(C, D, false, true);
    const uint32_t id_sink = idesc_bf16_f32(C, p.sk, false, false);
    // Descriptors of the first buffers; tiles and K steps add to their address field (16-byte units).
    const uint64_t d_own = smem_desc_sw128(cx.sbase + L::OFF_OWN, 16, 1024),
                   d_a = smem_desc_sw128(cx.sbase + L::OFF_A, 16, 1024), d_b = smem_desc_sw128(cx.sbase + L::OFF_B, 16, 1024),
                   m_a = smem_desc_sw128(cx.sbase + L::OFF_A, L::BLOCK, 1024),
                   m_b = smem_desc_sw128(cx.sbase + L::OFF_B, L::BLOCK, 1024),
                   m_a_sink = smem_desc_sw128(cx.sbase + L::OFF_A, p.sk * 128u, 1024);
    constexpr uint32_t TILE16 = L::TILE >> 4, BLOCK16 = L::BLOCK >> 4;
    bool ok = true;
    // D = own0 A^T (which 0: S) or own1 B^T (1: X) of ring step g and the unit's own buffer ob.
    const auto pair = [&](int which, int g, int ob, bool sink, bool final) {
        const int st = g % L::STAGES;
        const uint32_t ph = (g / L::STAGES) & 1;
        ok = ok && gwait_warp(cx, (which ? GB_BF : GB_AF) + st, ph);
        if (!ok) return;
        tc_fence_after();
        const uint64_t a = d_own + (ob * 2 + which) * TILE16, b = (which ? d_b : d_a) + st * TILE16;
        const uint32_t dst = tmem + (which ? L::COL_X : L::COL_S + (DKV ? 0 : 128 * (g & 1)));
        if (elect_one()) {
            if (sink) {
                for (int k = 0; k < D / 16; ++k)
                    mma_bf16(dst, a + (k >> 2) * BLOCK16 + (k & 3) * 2, b + (k >> 2) * p.sk * 8 + (k & 3) * 2, id_sink, k > 0);
            } else {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_bf16(dst, a + ((k >> 2) * BLOCK16 + (k & 3) * 2), b + ((k >> 2) * BLOCK16 + (k & 3) * 2), id_s, k > 0);
            }
            mma_commit(&cx.bars[which ? GB_XF : GB_SF + (DKV ? 0 : (g & 1))]);
            if (!DKV && which) mma_commit(&cx.bars[GB_BE + st]);             // V is read by X only
            if (which && final) mma_commit(&cx.bars[GB_OWNE + ob]);          // S went before
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
            for (int k = 1; k < C / 16; ++k) mma_bf16_ts(tmem + acc, tmem + src + 16 * k, b + k * 128, id_acc, 1u);
        }
    };
    const auto to_unit = [&](Walk& wk, int u) {              // the next unit with steps
        for (wk.start(p, u); wk.u < p.units && !wk.some; wk.start(p, wk.u + gridDim.x)) {}
    };
    const auto is_sink = [&](const Walk& wk) {
        if constexpr (DKV) return false;
        else return wk.t < 0;
    };
    Walk wk;
    to_unit(wk, blockIdx.x);
    int g = 0, nu = 0;
    if (wk.u < p.units) {
        ok = gwait_warp(cx, GB_OWNF, 0);
        pair(0, 0, 0, is_sink(wk), wk.last());
        pair(1, 0, 0, is_sink(wk), wk.last());
    }
    bool first = true;
    while (ok && wk.u < p.units) {
        const int st = g % L::STAGES, ob = nu % L::OWN;
        const bool sink = is_sink(wk), final = wk.last();
        // The step after this one, in this unit or the next.
        Walk nx = wk;
        if (final) to_unit(nx, wk.u + gridDim.x);
        else nx.next();
        const bool more = nx.u < p.units;
        const int nob = final ? (nu + 1) % L::OWN : ob;
        const bool nfinal = more && nx.last(), nsink = more && is_sink(nx);
        // The next unit's S can go early only into own tiles of another buffer.
        const bool early = more && (!final || L::OWN > 1);
        const auto enter = [&]() { if (final) ok = ok && gwait_warp(cx, GB_OWNF + nob, ((nu + 1) / L::OWN) & 1); };
        if constexpr (DKV) {
            ok = ok && gwait_warp(cx, GB_PF, g & 1);
            if (ok && first && nu > 0) ok = gwait_warp(cx, GB_ACCE, (nu - 1) & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                product(L::COL_ACC, L::COL_S, m_b + st * TILE16, false, first);          // dV += P dY
                mma_commit(&cx.bars[GB_BE + st]);
            }
            __syncwarp();
            if (early) {
                enter();
                pair(0, g + 1, nob, false, nfinal);
            }
            ok = ok && gwait_warp(cx, GB_DF, g & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                product(L::COL_ACC + D, L::COL_X, m_a + st * TILE16, false, first);      // dK += dS Q
                mma_commit(&cx.bars[GB_AE + st]);
                if (final) mma_commit(&cx.bars[GB_ACCF]);
            }
            __syncwarp();
        } else {
            if (early) {
                enter();
                pair(0, g + 1, nob, nsink, nfinal);
            }
            ok = ok && gwait_warp(cx, GB_DF, g & 1);
            if (ok && first && nu > 0) ok = gwait_warp(cx, GB_ACCE, (nu - 1) & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                product(L::COL_ACC, L::COL_X, (sink ? m_a_sink : m_a) + st * TILE16, sink, first);   // dQ += dS K
                mma_commit(&cx.bars[GB_AE + st]);
                if (final) mma_commit(&cx.bars[GB_ACCF]);
            }
            __syncwarp();
        }
        if (more && !early) {
            enter();
            pair(0, g + 1, nob, nsink, nfinal);
        }
        if (more) pair(1, g + 1, nob, nsink, nfinal);
        first = final;
        if (final) ++nu;
        ++g;
        wk = nx;
    }
    // Every MMA has completed: the last unit's accumulators are the last commit.
    if (ok && nu > 0) gwait_warp(cx, GB_ACCF, (nu - 1) & 1);
    if (g > 0) gdrain(cx, GB_AE + (g - 1) % L::STAGES, ((g - 1) / L::STAGES) & 1);
}

// ------------------------------------------------------------------ rows (warps 0-15)

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

// Rows [r0, r1) of a swizzled tile of D columns set to zero by all row threads.
template <int D>
__device__ __forceinline__ void zero_rows(uint32_t tile, uint32_t blk, int r0, int r1, int r, int cg) {
    if (r >= r0 && r < r1) {
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
            st_shared_v4(tile + h * blk + r * 128 + 32 * cg, make_uint4(0, 0, 0, 0));
            st_shared_v4(tile + h * blk + r * 128 + 32 * cg + 16, make_uint4(0, 0, 0, 0));
        }
    }
    fence_proxy_async_smem();
    __syncwarp();
}

// Reads D / 4 columns (this thread's share) of an accumulator row, scales them and hands
// over 8 at a time.
template <int D, typename F>
__device__ __forceinline__ void read_out(uint32_t taddr, int cg, float scale, F&& put) {
#pragma unroll
    for (int q = 0; q < D / 64; ++q) {
        float o[16];
        tmem_ld16(taddr + D / 4 * cg + 16 * q, o);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] *= scale;
        put(D / 4 * cg + 16 * q, o);
        put(D / 4 * cg + 16 * q + 8, o + 8);
        __syncwarp();
    }
}

__device__ __forceinline__ __nv_bfloat16* row_ptr(const View& v, int b, int h, int n) {
    return static_cast<__nv_bfloat16*>(v.p) + b * v.sb + h * v.sh + n * v.sn;
}

template <int D>
__device__ __forceinline__ void dq_rows(const BwdCtx& cx, const BwdParams& p, uint32_t tmem, int cg, int wq, int lane) {
    using L = BwdLayout<D, false>;
    const int r = wq * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    int g = 0, nu = 0;
    DqWalk wk;
    for (wk.start(p, blockIdx.x); wk.u < p.units; wk.start(p, wk.u + gridDim.x)) {
        const int i0 = wk.tile * C, i = i0 + r;
        const bool live = i < wk.len;
        if (wk.some) {
            // delta: each thread a quarter of the row's channels, summed over the four.
            const size_t row = (size_t)wk.b * p.Hq + wk.h;
            float part = 0.f, nl = 0.f;
            if (live) {
                const uint4* a = reinterpret_cast<const uint4*>(row_ptr(p.dy, wk.b, wk.h, i) + D / 4 * cg);
                const uint4* b = reinterpret_cast<const uint4*>(row_ptr(p.y, wk.b, wk.h, i) + D / 4 * cg);
#pragma unroll
                for (int q = 0; q < D / 32; ++q) {
                    const uint4 x = __ldg(a + q), z = __ldg(b + q);
                    const uint32_t wa[4] = {x.x, x.y, x.z, x.w}, wb[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        part = fmaf(__uint_as_float(wa[e] << 16), __uint_as_float(wb[e] << 16), part);
                        part = fmaf(__uint_as_float(wa[e] & 0xFFFF0000u), __uint_as_float(wb[e] & 0xFFFF0000u), part);
                    }
                }
                nl = -p.lse[row * p.N + i] * kLog2e;
            }
            const uint32_t red = cx.sbase + L::OFF_RED + (nu & 1) * 4 * C * 4 + 4 * r;
            st_shared_f32(red + cg * C * 4, part);
            __syncwarp();
            if (lane == 0) mbar_arrive(&cx.bars[GB_RED]);
            if (!gwait(cx, GB_RED, nu & 1)) return;
            float delta = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) delta += ld_shared_f32(red + q * C * 4);
            if (cg == 0) {
                p.nl2[row * p.npad + i] = nl;
                p.delta[row * p.npad + i] = delta;
            }
            for (;; ++g) {
                const bool sink = wk.t < 0;
                const int j0 = sink ? 0 : wk.t * C, c0 = 32 * cg;
                uint32_t vis = ~0u;
                if (sink || j0 + C > i0 || j0 < i0 + C - p.w) {
                    const int hi = (sink ? p.n_sink : i - j0 + 1) - c0, lo = (sink ? 0 : i - p.w + 1 - j0) - c0;
                    vis = low_bits(hi) & (~low_bits(lo) | low_bits((j0 == 0 ? p.n_sink : 0) - c0));
                }
                const WordMask mask(vis);
                const bool any = mask.kind != WordMask::kNone;   // for some row of this warp
                if (!gwait(cx, GB_SF + (g & 1), (g >> 1) & 1)) return;
                tc_fence_after();
                float pr[32];
                if (any) {
                    tmem_ld32(tl + L::COL_S + 128 * (g & 1) + c0, pr);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; e += 4) add_scaled(pr + e, p.c, nl, nl, nl, nl);
#pragma unroll
                    for (int e = 0; e < 32; ++e) pr[e] = ex2(pr[e]);
                    mask.apply(pr, 0.f);
                }
                // K rows that no dS may meet: padding in the tile of the sequence's end, tokens
                // after the sinks in their block.
                const int k0 = sink ? p.n_sink : wk.len - j0, k1 = sink ? p.sk : min(C, p.N - j0);
                if ((sink || wk.last()) && k0 < k1) {
                    const int st = g % L::STAGES;
                    if (!gwait(cx, GB_AF + st, (g / L::STAGES) & 1)) return;
                    zero_rows<D>(cx.sbase + L::OFF_A + st * L::TILE, sink ? p.sk * 128u : L::BLOCK, k0, k1, r, cg);
                }
                if (!gwait(cx, GB_XF, g & 1)) return;
                tc_fence_after();
                float x[32];
                if (any) {
                    tmem_ld32(tl + L::COL_X + c0, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; e += 2) dscore(x[e], x[e + 1], pr[e], pr[e + 1], delta, delta);
                    mask.apply(x, 0.f);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = 0.f;
                }
                put32(tl + L::COL_X + c0, x);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&cx.bars[GB_DF]);
                if (wk.last()) break;
                wk.next();
            }
            ++g;
            if (!gwait(cx, GB_ACCF, nu & 1)) return;
            tc_fence_after();
        }
        __nv_bfloat16* out = row_ptr(p.dq, wk.b, wk.h, i);
        if (wk.some) {
            read_out<D>(tl + L::COL_ACC, cg, p.scale, [&](int col, const float* o) {
                if (i < p.N)
                    *reinterpret_cast<uint4*>(out + col) = live ? pack_bf16x8(o) : make_uint4(0, 0, 0, 0);
            });
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&cx.bars[GB_ACCE]);
            ++nu;
        } else if (i < p.N) {
#pragma unroll
            for (int q = 0; q < D / 32; ++q)
                *reinterpret_cast<uint4*>(out + D / 4 * cg + 8 * q) = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
    }
}

template <int D>
__device__ __forceinline__ void dkv_rows(const BwdCtx& cx, const BwdParams& p, uint32_t tmem, int cg, int wq, int lane) {
    using L = BwdLayout<D, true>;
    const int r = wq * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const int c0 = 32 * cg;
    int g = 0, nu = 0;
    KvWalk wk;
    for (wk.start(p, blockIdx.x); wk.u < p.units; wk.start(p, wk.u + gridDim.x)) {
        const int j0 = wk.kt * C, j = j0 + r;
        const bool chunk = wk.chunk >= 0;
        if (wk.some) {
            for (;; ++g) {
                const int i0 = wk.t * C, st = g % L::STAGES;
                const uint32_t ph = (g / L::STAGES) & 1;
                // Visible queries of this key: [j, j + w) in a band unit, [j + w, ..) for a sink
                // in a chunk; none past the sequence's end.
                uint32_t vis = ~0u;
                if (chunk || i0 < j0 + C || i0 + C > j0 + p.w || i0 + C > wk.len) {
                    const int first = chunk ? (r < p.n_sink ? j + p.w : 0x7fffffff) : j;
                    const int end = chunk ? wk.len : min(wk.len, j + p.w);
                    vis = low_bits(end - i0 - c0) & ~low_bits(first - i0 - c0);
                }
                const WordMask mask(vis);
                const bool any = mask.kind != WordMask::kNone;   // for some row of this warp
                if (!gwait(cx, GB_SF, g & 1)) return;
                if (!gwait(cx, GB_AF + st, ph)) return;
                tc_fence_after();
                const uint32_t rows = cx.sbase + L::OFF_ROW + st * 2 * C * 4 + 4 * c0;
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
                if (i0 + C > wk.len && wk.len < p.N) {
                    if (!gwait(cx, GB_BF + st, ph)) return;
                    zero_rows<D>(cx.sbase + L::OFF_A + st * L::TILE, L::BLOCK, wk.len - i0, C, r, cg);
                    zero_rows<D>(cx.sbase + L::OFF_B + st * L::TILE, L::BLOCK, wk.len - i0, C, r, cg);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&cx.bars[GB_PF]);
                if (!gwait(cx, GB_XF, g & 1)) return;
                tc_fence_after();
                float x[32];
                if (any) {
                    tmem_ld32(tl + L::COL_X + c0, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        float d[4];
                        ld_shared_f4(rows + C * 4 + 4 * e, d);
                        dscore(x[e], x[e + 1], pr[e], pr[e + 1], d[0], d[1]);
                        dscore(x[e + 2], x[e + 3], pr[e + 2], pr[e + 3], d[2], d[3]);
                    }
                    mask.apply(x, 0.f);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = 0.f;
                }
                put32(tl + L::COL_X + c0, x);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&cx.bars[GB_DF]);
                if (wk.last()) break;
                wk.next();
            }
            ++g;
            if (!gwait(cx, GB_ACCF, nu & 1)) return;
            tc_fence_after();
        }
        // Sink rows go to partials (slot 0: the sink tile's band unit, 1 + c: chunk c).
        const bool sink = p.sp.chunks > 0 && j < p.n_sink;
        const bool store = j < p.N && (!chunk || sink), zero = !wk.some || j >= wk.len;
        float* part = p.partial + sink_partial_offset(p.sp, wk.b * p.Hkv + wk.hk, wk.chunk + 1, D) + (size_t)r * D;
        __nv_bfloat16* ok = row_ptr(p.dk, wk.b, wk.hk, j);
        __nv_bfloat16* ov = row_ptr(p.dv, wk.b, wk.hk, j);
        const auto put = [&](bool value, int col, const float* o) {
            if (!store) return;
            if (sink) {
                float* q = part + (value ? (size_t)p.sp.rows * D : 0) + col;
                *reinterpret_cast<float4*>(q) = zero ? make_float4(0, 0, 0, 0) : make_float4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<float4*>(q + 4) = zero ? make_float4(0, 0, 0, 0) : make_float4(o[4], o[5], o[6], o[7]);
            } else {
                *reinterpret_cast<uint4*>((value ? ov : ok) + col) = zero ? make_uint4(0, 0, 0, 0) : pack_bf16x8(o);
            }
        };
        if (wk.some) {
            read_out<D>(tl + L::COL_ACC, cg, 1.0f, [&](int col, const float* o) { put(true, col, o); });
            read_out<D>(tl + L::COL_ACC + D, cg, p.scale, [&](int col, const float* o) { put(false, col, o); });
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&cx.bars[GB_ACCE]);
            ++nu;
        } else {
            const float none[8] = {};
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
                put(true, D / 4 * cg + 8 * q, none);
                put(false, D / 4 * cg + 8 * q, none);
            }
        }
        __syncwarp();
    }
}

template <int D, bool DKV>
__global__ void __launch_bounds__(kThreads, 1)
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
    const BwdCtx cx{sbase, bars, abort_flag, p.status};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int b = 0; b < GB_NUM; ++b)
            mbar_init(&bars[b], b == GB_PF || b == GB_DF || b == GB_ACCE || b == GB_RED ? kRowWarps : 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == kRowWarps + 1) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();                                  // inputs and workspace may come from earlier kernels
    using Walk = typename std::conditional<DKV, KvWalk, DqWalk>::type;
    if (warp == kRowWarps) {
        if (lane == 0) bwd_load<D, DKV, Walk>(cx, p, BwdMaps{&own0, &own1, &ma, &mb, &ma_sink, &mb_sink});
    } else if (warp == kRowWarps + 1) {
        if (!(p.debug & DEBUG_SKIP_MMA)) bwd_mma<D, DKV, Walk>(cx, p, tmem);
    } else if (warp < kRowWarps) {
        if constexpr (DKV) dkv_rows<D>(cx, p, tmem, warp >> 2, warp & 3, lane);
        else dq_rows<D>(cx, p, tmem, warp >> 2, warp & 3, lane);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kRowWarps + 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
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
    return launch_pdl(kern, dim3(std::min(p.units, num_sms)), dim3(kThreads), L::SMEM_BYTES, stream, own0, own1, ma, mb,
                      mas, mbs, p);
}

size_t padded_rows(int N) { return (size_t)(N + C - 1) / C * C; }

template <int D>
cudaError_t run(const SinkArgs& a, int num_sms, cudaStream_t stream) {
    BwdParams p{};
    p.lengths = a.lengths, p.lse = a.lse, p.status = a.status, p.debug = a.debug;
    p.y = a.y, p.dy = a.dy, p.dq = a.dq, p.dk = a.dk, p.dv = a.dv;
    p.B = a.B, p.Hq = a.Hq, p.Hkv = a.Hkv, p.N = a.N, p.w = a.w, p.n_sink = a.n_sink;
    p.sk = std::max(16, (a.n_sink + 15) / 16 * 16);
    p.nt = (a.N + C - 1) / C;
    p.npad = (int)padded_rows(a.N);
    p.c = a.scale * kLog2e;
    p.scale = a.scale;
    p.sp = sink_split(a.Hq, a.Hkv, a.N, a.w, a.n_sink, C);
    const size_t vec = (size_t)a.B * a.Hq * p.npad;
    p.nl2 = static_cast<float*>(a.workspace);
    p.delta = p.nl2 + vec;
    p.partial = p.delta + vec;
    CUtensorMap mq, mk, mv, mg, mks, mvs;
    if (!heads_map(&mq, a.q, a, a.Hq, C) || !heads_map(&mg, a.dy, a, a.Hq, C) || !heads_map(&mk, a.k, a, a.Hkv, C) || !heads_map(&mv, a.v, a, a.Hkv, C) ||
        !heads_map(&mks, a.k, a, a.Hkv, p.sk) || !heads_map(&mvs, a.v, a, a.Hkv, p.sk))
        return cudaErrorInvalidValue;
    p.units = a.B * a.Hq * p.nt;
    cudaError_t e = launch<D, false>(mq, mg, mk, mv, mks, mvs, p, num_sms, stream);
    p.units = a.B * a.Hkv * p.sp.units();
    if (e == cudaSuccess) e = launch<D, true>(mk, mv, mq, mg, mq, mg, p, num_sms, stream);
    if (e == cudaSuccess && p.sp.chunks > 0) e = launch_sink_join<__nv_bfloat16>(a, p.sp, p.partial, stream);
    return e;
}

}  // namespace

size_t sink_backward_workspace_tc(int B, int Hq, int Hkv, int N, int d, int w, int n_sink) {
    const SinkSplit sp = sink_split(Hq, Hkv, N, w, n_sink, C);
    return (2 * (size_t)B * Hq * padded_rows(N) + sink_partial_offset(sp, B * Hkv, 0, d)) * sizeof(float);
}

cudaError_t launch_sink_backward_tc(const SinkArgs& a, int num_sms, cudaStream_t stream) {
    return a.d == 64 ? run<64>(a, num_sms, stream) : run<128>(a, num_sms, stream);
}

}  // namespace based
