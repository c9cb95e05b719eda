// Prompt form of the sliding-window attention with sink tokens on the tensor cores (bf16)
// for narrow windows.
//
// A window of a few tiles gives a query tile so few steps that the wide kernel
// (sink_fwd_tc.cu) waits through the latency of each: tensor core, rows, tensor core,
// output. Here a block walks tiles of 128 queries in steps of 64 keys and is small enough
// that several blocks share an SM (four at d = 64, two at d = 128: S takes 64 and O d
// columns of tensor memory) and cover each other's waits. The arithmetic is the same: S
// = Q K^T, one thread per row forms the weights (bf16, over S), O += P V; the sink
// tokens come as a short block of their own where the window has left them behind.
// 8 x 16 heads x 2048 x 64, w = 64, 4 sinks: 39 us without the cache (134 MB, 3.4 TB/s of
// 6.55), 35 without sinks; w = 512: 82 us. Latency bounds it: four short steps per tile, of a product, the
// weights, a product. Rescaling and masks as in the wide kernel.
// Roles (192 threads): warps 0-3 the rows, warp 4 the TMA loads, warp 5 TMEM
// allocation and the MMAs.
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

constexpr int C = 128;                       // queries of a block
constexpr int W = 64;                        // keys of a step
constexpr int kThreads = 192;

template <int D>
struct NarrowLayout {
    static constexpr uint32_t QBLOCK = C * 128, KBLOCK = W * 128;   // 64 columns, 128-byte swizzle
    static constexpr uint32_t QTILE = C * D * 2, KTILE = W * D * 2;
    static constexpr int STAGES = 2;                         // K and V tiles each
    static constexpr uint32_t OFF_Q = 0;                     // Q, at the end of a unit its outputs
    static constexpr uint32_t OFF_K = OFF_Q + QTILE;
    static constexpr uint32_t OFF_V = OFF_K + STAGES * KTILE;
    static constexpr uint32_t OFF_BAR = OFF_V + STAGES * KTILE;
    static constexpr uint32_t SMEM_BYTES = OFF_BAR + 256 + 1024;
    static constexpr int BLOCKS_PER_SM = D == 64 ? 4 : 2;
    static constexpr uint32_t TMEM_COLS = D == 64 ? 128 : 256;
    static_assert(BLOCKS_PER_SM * (SMEM_BYTES + 1024) <= 228 * 1024, "shared memory of an SM");
    static_assert(BLOCKS_PER_SM * TMEM_COLS <= 512, "tensor memory of an SM");
    static_assert(STAGES == 2, "barriers of the ring");
    static constexpr uint32_t COL_S = 0, COL_O = 64;
};

enum {
    NB_QF = 0,                // TMA: Q landed
    NB_QE,                    // the store's thread: Q's place is free
    NB_KF,                    // [2] TMA: K of stage s landed
    NB_VF = NB_KF + 2,        // [2]
    NB_KE = NB_VF + 2,        // [2] MMA commit: K of stage s read
    NB_VE = NB_KE + 2,        // [2]
    NB_SF = NB_VE + 2,        // MMA commit: S of the step ready (and O at rest)
    NB_PF,                    // row warps: P of the step written
    NB_OF,                    // MMA commit: O of the unit complete
    NB_OE,                    // row warps: O read out
    NB_YF,                    // row warps: outputs staged
    NB_NUM
};

struct NarrowParams {
    const int64_t* lengths;
    View q, k, v, y;
    float* lse;
    unsigned* status;
    int B, Hq, Hkv, N, w, n_sink, sk;        // sk: n_sink rounded up to 16
    FastDiv by_nt, by_hq, by_group;
    int nt, units;
    float c, scale;                          // c: scale * log2(e)
    unsigned debug;
    int fill;                                // the cache's fill follows
};

// One tile of one head, its steps: the sink block, if the window has left it, then key
// tiles lo .. hi. Head-major, so that blocks that run together share key tiles in L2.
struct NarrowUnit {
    int b, h, hk, i0, len, lo, steps;
    bool sinks;
    __device__ __forceinline__ NarrowUnit(const NarrowParams& p, int u, unsigned* status) {
        const int bh = p.by_nt.div(u);
        i0 = (u - bh * p.nt) * C;
        b = p.by_hq.div(bh);
        h = bh - b * p.Hq;
        hk = p.by_group.div(h);
        len = p.N;
        if (p.lengths != nullptr) {
            const int64_t n = p.lengths[b];
            if ((n < 0 || n > p.N) && status != nullptr) atomicOr(status, DEV_ERR_RANGE);
            len = n < 0 ? 0 : n > p.N ? p.N : (int)n;
        }
        lo = max(0, i0 - p.w + 1) / W;
        sinks = p.n_sink > 0 && lo > 0;
        steps = i0 < len ? (min(i0 + C, len) - 1) / W - lo + 1 + (sinks ? 1 : 0) : 0;
    }
    __device__ __forceinline__ bool is_sink(int j) const { return sinks && j == 0; }
    __device__ __forceinline__ int key(int j) const { return is_sink(j) ? 0 : (lo + j - (sinks ? 1 : 0)) * W; }
};

struct NarrowCtx {
    uint32_t sbase;
    uint64_t* bars;
    volatile int* abort_flag;
    volatile int* redo;                      // some row came out non-finite
    unsigned* status;
    __device__ __forceinline__ bool wait(int bar, uint32_t parity) const {
        return mbar_wait(&bars[bar], parity, abort_flag, status);
    }
    __device__ __forceinline__ bool wait_joint(int bar, uint32_t parity) const {
        return mbar_wait_joint(&bars[bar], parity, abort_flag, status);
    }
    __device__ __forceinline__ bool wait_warp(int bar, uint32_t parity) const {
        return mbar_wait_warp(&bars[bar], parity, abort_flag, status);
    }
    // After an abort: wait (bounded) for this thread's own last asynchronous work.
    __device__ __forceinline__ void drain(int bar, uint32_t parity) const {
        if (!*abort_flag || bar < 0) return;
        const uint64_t t0 = global_ns();
        while (!mbar_try_wait(&bars[bar], parity) && global_ns() - t0 < kWaitLimitNs) {}
    }
};

// ------------------------------------------------------------------ TMA loads (warp 4, lane 0)
template <int D>
__device__ __forceinline__ void narrow_load(const NarrowCtx& cx, const NarrowParams& p, const CUtensorMap* mq,
                                            const CUtensorMap* mk, const CUtensorMap* mv, const CUtensorMap* mks,
                                            const CUtensorMap* mvs) {
    using L = NarrowLayout<D>;
    int g = 0, nu = 0, last = -1;
    uint32_t lastp = 0;
    const auto tile = [&](int bar, uint32_t dst, const CUtensorMap* m, uint32_t blk, int row, int head, int b) {
        mbar_expect_tx(&cx.bars[bar], blk * (D / 64));
#pragma unroll
        for (int x = 0; x < D / 64; ++x) tma_load_4d(cx.sbase + dst + x * blk, m, &cx.bars[bar], 64 * x, row, head, b);
        last = bar;
    };
    for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
        const NarrowUnit un(p, u, p.status);
        if (un.steps == 0) continue;
        for (int j = 0; j < un.steps; ++j, ++g) {
            const int st = g % L::STAGES;
            const uint32_t ph = (g / L::STAGES) & 1;
            const bool sink = un.is_sink(j);
            const uint32_t blk = sink ? p.sk * 128u : L::KBLOCK;
            if (g >= L::STAGES && !cx.wait(NB_KE + st, ph ^ 1)) { cx.drain(last, lastp); return; }
            tile(NB_KF + st, L::OFF_K + st * L::KTILE, sink ? mks : mk, blk, un.key(j), un.hk, un.b);
            lastp = ph;
            if (j == 0) {
                if (nu > 0 && !cx.wait(NB_QE, (nu - 1) & 1)) { cx.drain(last, lastp); return; }
                tile(NB_QF, L::OFF_Q, mq, L::QBLOCK, un.i0, un.h, un.b);
                lastp = nu++ & 1;
            }
            if (g >= L::STAGES && !cx.wait(NB_VE + st, ph ^ 1)) { cx.drain(last, lastp); return; }
            tile(NB_VF + st, L::OFF_V + st * L::KTILE, sink ? mvs : mv, blk, un.key(j), un.hk, un.b);
            lastp = ph;
        }
    }
    cx.drain(last, lastp);
}

// ------------------------------------------------------------------ MMAs (warp 5)
template <int D>
__device__ __forceinline__ void narrow_mma(const NarrowCtx& cx, const NarrowParams& p, uint32_t tmem) {
    using L = NarrowLayout<D>;
    constexpr uint32_t id_s = idesc_bf16_f32(C, W, false, false), id_o = idesc_bf16_f32(C, D, false, true);
    const uint32_t id_sink = idesc_bf16_f32(C, p.sk, false, false);
    const uint64_t dq = smem_desc_sw128(cx.sbase + L::OFF_Q, 16, 1024), dk = smem_desc_sw128(cx.sbase + L::OFF_K, 16, 1024),
                   dv = smem_desc_sw128(cx.sbase + L::OFF_V, L::KBLOCK, 1024),
                   dv_sink = smem_desc_sw128(cx.sbase + L::OFF_V, p.sk * 128u, 1024);
    const uint32_t ts = tmem + L::COL_S, to = tmem + L::COL_O;
    int g = 0, nu = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
        const NarrowUnit un(p, u, nullptr);
        if (un.steps == 0) continue;
        for (int j = 0; ok && j <= un.steps; ++j) {
            if (j > 0) {                                     // O += P V of step j - 1
                const int st = (g + j - 1) % L::STAGES;
                ok = cx.wait_warp(NB_VF + st, ((g + j - 1) / L::STAGES) & 1);
                if (ok && j == 1 && nu > 0) ok = cx.wait_warp(NB_OE, (nu - 1) & 1);
                ok = ok && cx.wait_warp(NB_PF, (g + j - 1) & 1);
                if (!ok) break;
                tc_fence_after();
                const bool sink = un.is_sink(j - 1);
                const uint64_t v = (sink ? dv_sink : dv) + st * (L::KTILE >> 4);
                if (elect_one()) {
                    if (sink) {
                        for (int k = 0; k < p.sk / 16; ++k) mma_bf16_ts(to, ts + 8 * k, v + k * 128, id_o, k > 0);
                    } else {
                        mma_bf16_ts(to, ts, v, id_o, j > 1);
#pragma unroll
                        for (int k = 1; k < W / 16; ++k) mma_bf16_ts(to, ts + 8 * k, v + k * 128, id_o, 1u);
                    }
                    mma_commit(&cx.bars[NB_VE + st]);
                    if (j == un.steps) mma_commit(&cx.bars[NB_OF]);
                }
                __syncwarp();
            }
            if (j < un.steps) {                              // S = Q K^T of step j
                const int st = (g + j) % L::STAGES;
                ok = cx.wait_warp(NB_KF + st, ((g + j) / L::STAGES) & 1);
                if (ok && j == 0) ok = cx.wait_warp(NB_QF, nu & 1);
                if (!ok) break;
                tc_fence_after();
                const uint64_t k0 = dk + st * (L::KTILE >> 4);
                if (elect_one()) {
                    if (un.is_sink(j)) {
                        for (int k = 0; k < D / 16; ++k)
                            mma_bf16(ts, dq + (k >> 2) * (L::QBLOCK >> 4) + (k & 3) * 2,
                                     k0 + (k >> 2) * p.sk * 8 + (k & 3) * 2, id_sink, k > 0);
                    } else {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            mma_bf16(ts, dq + ((k >> 2) * (L::QBLOCK >> 4) + (k & 3) * 2),
                                     k0 + ((k >> 2) * (L::KBLOCK >> 4) + (k & 3) * 2), id_s, k > 0);
                    }
                    mma_commit(&cx.bars[NB_SF]);
                    mma_commit(&cx.bars[NB_KE + st]);
                }
                __syncwarp();
            }
        }
        g += un.steps;
        ++nu;
    }
    // Every MMA has completed: O of the last unit is the last commit.
    if (ok && nu > 0) cx.wait_warp(NB_OF, (nu - 1) & 1);
    if (nu > 0) cx.drain(NB_OF, (nu - 1) & 1);
}

// ------------------------------------------------------------------ rows (warps 0-3)
template <int D>
__device__ __forceinline__ void narrow_rows(const NarrowCtx& cx, const NarrowParams& p, const CUtensorMap* my, uint32_t tmem,
                                            int warp, int lane) {
    using L = NarrowLayout<D>;
    const int r = warp * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const uint32_t ts = tl + L::COL_S, to = tl + L::COL_O;
    int g = 0, nu = 0;
    for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
        const NarrowUnit un(p, u, nullptr);
        const int i = un.i0 + r;
        float m = -INFINITY, l0 = 0.f, l1 = 0.f;             // m: of the scores times c
        for (int j = 0; j < un.steps; ++j, ++g) {
            const bool sink = un.is_sink(j);
            const int j0 = un.key(j);
            // Visible columns: [cl, ch) are inside the window, and the sinks of tile 0 stay
            // visible below it.
            uint32_t vis[2] = {~0u, ~0u};
            if (sink || j0 + W > un.i0 + 1 || j0 < un.i0 + C - p.w) {
                const int ch = sink ? p.n_sink : i - j0 + 1, cl = sink ? 0 : i - p.w + 1 - j0;
                const int cs = j0 == 0 ? p.n_sink : 0;
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    vis[q] = low_bits(ch - 32 * q) & (~low_bits(cl - 32 * q) | low_bits(cs - 32 * q));
            }
            const WordMask mask[2] = {WordMask(vis[0]), WordMask(vis[1])};
            if (!cx.wait_joint(NB_SF, g & 1)) return;
            tc_fence_after();
            float mt = -INFINITY;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (mask[q].kind == WordMask::kNone) continue;   // no row of this warp sees these columns
                float sv[32];
                tmem_ld32(ts + 32 * q, sv);
                tmem_ld_wait();
                mask[q].apply(sv, -INFINITY);
                mt = fmaxf(mt, max32(sv));
            }
            mt *= p.c;                                       // -inf stays: c > 0
            const bool grown = mt > m + 8.0f;
            if (__any_sync(0xffffffffu, grown)) {
                const float al = grown ? ex2(m - mt) : 1.0f; // 0 the first time
                l0 *= al;
                l1 *= al;
                if (grown) m = mt;
                if (j > 0) scale_row<D>(to, al);
            }
            const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int q = 0; q < 2; ++q) {                    // the weights overlay scores that are read already
                uint32_t pb[16];
                if (mask[q].kind != WordMask::kNone) {
                    float sv[32];
                    tmem_ld32(ts + 32 * q, sv);
                    tmem_ld_wait();
                    mask[q].apply(sv, -INFINITY);
                    weights32(sv, p.c, mu, pb, l0, l1);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) pb[e] = 0u;
                }
                tmem_st16(ts + 16 * q, pb);
            }
            // Rows of V that no weight may meet: padding in the tile of the sequence's end (the
            // tensor's own end is zero-filled), tokens after the sinks in their block.
            const int v0 = sink ? p.n_sink : un.len - j0, v1 = sink ? p.sk : min(W, p.N - j0);
            if (v0 < v1) {
                const int st = g % L::STAGES;
                if (!cx.wait_joint(NB_VF + st, (g / L::STAGES) & 1)) return;
                const uint32_t blk = sink ? p.sk * 128u : L::KBLOCK;
                const uint32_t row = cx.sbase + L::OFF_V + st * L::KTILE + (r & 63) * 128 + (r >> 6) * 64;
                if ((r & 63) >= v0 && (r & 63) < v1) {       // two threads per row
#pragma unroll
                    for (int x = 0; x < D / 64; ++x)
#pragma unroll
                        for (int q = 0; q < 4; ++q) st_shared_v4(row + x * blk + 16 * q, make_uint4(0, 0, 0, 0));
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&cx.bars[NB_PF]);
        }
        // ---- outputs
        const bool on = un.steps > 0, live = i < un.len;
        const float l = l0 + l1;
        const float inv = live ? 1.0f / l : 0.f;
        if (p.lse != nullptr && i < p.N)
            p.lse[((size_t)un.b * p.Hq + un.h) * p.N + i] = live ? m * kLn2 + logf(l) : -INFINITY;
        if (on) {
            if (!cx.wait_joint(NB_OF, nu & 1)) return;
            tc_fence_after();
            // Over Q in shared memory (every product has completed), out by TMA.
            float odd = 0.f;                                 // NaN where an output is not finite
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
                float o[32];
                tmem_ld32(to + 32 * x, o);
                tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        v[e] = live ? o[8 * q + e] * inv : 0.f;
                        odd = fmaf(v[e], 0.f, odd);
                    }
                    st_shared_v4(cx.sbase + L::OFF_Q + (x >> 1) * L::QBLOCK + sw128_offset(r, 4 * (x & 1) + q),
                                 pack_bf16x8(v));
                }
            }
            if (live && odd != 0.f) *cx.redo = 1;
            tc_fence_before();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&cx.bars[NB_OE]);                // O may be overwritten
                mbar_arrive(&cx.bars[NB_YF]);
            }
            if (warp == 0) {                                 // whole: its lanes leave together or not at all
                if (!cx.wait_warp(NB_YF, nu & 1)) return;
                if (lane == 0) {
#pragma unroll
                    for (int x = 0; x < D / 64; ++x)
                        tma_store_4d(my, cx.sbase + L::OFF_Q + x * L::QBLOCK, 64 * x, un.i0, un.h, un.b);
                    bulk_commit();
                    bulk_wait_read_all();
                    mbar_arrive(&cx.bars[NB_QE]);
                }
            }
            __syncwarp();
            ++nu;
        } else if (i < p.N) {
            __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y.p) + un.b * p.y.sb + un.h * p.y.sh + i * p.y.sn;
#pragma unroll
            for (int q = 0; q < D / 8; ++q) *reinterpret_cast<uint4*>(y + 8 * q) = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
    }
    if (warp == 0 && lane == 0) bulk_wait_all();
}

// Non-finite rows of the block's units, again from their definition.
template <int D>
__device__ __noinline__ void narrow_redo(const NarrowParams& p, int warp) {
    for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
        const NarrowUnit un(p, u, nullptr);
        redo_rows<__nv_bfloat16, D>(p, un.b, un.h, un.hk, un.i0, C, un.len, un.lo * W, 0, warp, kThreads / 32);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, NarrowLayout<D>::BLOCKS_PER_SM)
sink_fwd_narrow_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mks,
                       const __grid_constant__ CUtensorMap mvs, const __grid_constant__ CUtensorMap my,
                       const __grid_constant__ NarrowParams p) {
    using L = NarrowLayout<D>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    unsigned char* smem = smem_raw + (sbase - raw);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_BAR + 8 * NB_NUM);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_BAR + 8 * NB_NUM + 4);
    const NarrowCtx cx{sbase, bars, abort_flag, abort_flag + 1, p.status};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int b = 0; b < NB_NUM; ++b) mbar_init(&bars[b], b == NB_PF || b == NB_OE || b == NB_YF ? 4 : 1);
        *abort_flag = 0;
        *cx.redo = 0;
        mbar_fence_init();
    }
    if (warp == 5) tmem_alloc(tmem_slot, L::TMEM_COLS);
    if (warp == 4 && lane == 0) {
        prefetch_tensormap(&mq);
        prefetch_tensormap(&mk);
        prefetch_tensormap(&mv);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();                                  // inputs may come from earlier kernels
    if (p.fill) grid_launch_dependents();                    // the cache's fill may start
    if (warp == 4) {
        if (lane == 0) narrow_load<D>(cx, p, &mq, &mk, &mv, &mks, &mvs);
    } else if (warp == 5) {
        if (!(p.debug & DEBUG_SKIP_MMA)) narrow_mma<D>(cx, p, tmem);
    } else {
        narrow_rows<D>(cx, p, &my, tmem, warp, lane);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, L::TMEM_COLS);
    }
    if (*cx.redo && !*abort_flag) narrow_redo<D>(p, warp);   // the outputs have landed
}

template <int D>
cudaError_t run(const SinkArgs& a, int num_sms, cudaStream_t stream) {
    using L = NarrowLayout<D>;
    NarrowParams p{};
    p.lengths = a.lengths, p.q = a.q, p.k = a.k, p.v = a.v, p.y = a.y, p.lse = a.lse, p.status = a.status, p.debug = a.debug, p.fill = a.fill;
    p.B = a.B, p.Hq = a.Hq, p.Hkv = a.Hkv, p.N = a.N, p.w = a.w, p.n_sink = a.n_sink;
    p.sk = std::max(16, (a.n_sink + 15) / 16 * 16);
    p.nt = (a.N + C - 1) / C;
    p.units = p.nt * a.B * a.Hq;
    p.by_nt = FastDiv(p.nt), p.by_hq = FastDiv(a.Hq), p.by_group = FastDiv(a.Hq / a.Hkv);
    // A scale of 0 (equal weights) becomes the least number, so that -inf times it stays -inf
    // and any finite score times it is next to 0.
    p.c = std::max(a.scale * kLog2e, std::numeric_limits<float>::denorm_min());
    p.scale = a.scale;
    CUtensorMap mq, mk, mv, mks, mvs, my;
    if (!heads_map(&mq, a.q, a, a.Hq, C) || !heads_map(&mk, a.k, a, a.Hkv, W) || !heads_map(&mv, a.v, a, a.Hkv, W) ||
        !heads_map(&mks, a.k, a, a.Hkv, p.sk) || !heads_map(&mvs, a.v, a, a.Hkv, p.sk) ||
        !heads_map(&my, a.y, a, a.Hq, C))
        return cudaErrorInvalidValue;
    auto kern = sink_fwd_narrow_kernel<D>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(std::min(p.units, num_sms * L::BLOCKS_PER_SM)), dim3(kThreads), L::SMEM_BYTES, stream, mq,
                      mk, mv, mks, mvs, my, p);
}

}  // namespace

cudaError_t launch_sink_prefill_narrow(const SinkArgs& a, int num_sms, cudaStream_t stream) {
    return a.d == 64 ? run<64>(a, num_sms, stream) : run<128>(a, num_sms, stream);
}

}  // namespace based
