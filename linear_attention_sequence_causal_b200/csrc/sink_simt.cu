// Sliding-window attention with sink tokens on the CUDA cores: forward, backward and
// the generation cache's fill. All arithmetic is fp32.
//
// visible(i) = { j <= i : j > i - w or j < n_sink }. A block owns 64 query rows of a
// head (forward, dQ) or 64 keys of a key/value head (dK, dV) and sweeps the 64-row
// tiles of the other side; its 256 threads form a 16 x 16 grid, each holding a 4 x 4
// piece of a score tile and 4 rows x d/16 columns of the accumulators, so every
// float4 from shared memory feeds 4 to 16 multiply-adds.
// The tiles of a query tile are the sink tile (when the window has left it behind)
// and the window's own tiles. For dK, dV the two kinds of pairs are apart: "band"
// units take j > i - w, and the pairs with the sink tokens outside the window, which
// every later query has, are cut into chunks of query tiles whose fp32 partials
// (with the sink tile's band partial) sink_join_kernel adds in a fixed order.
//
// The forward of 5 sequences (padded to 1337) x 8 heads (2 key/value) x 64, w = 200: 82 us;
// of all 5 in full 152 us: 18 TFLOP/s over the visible pairs, 28 over the tiles' pairs (w =
// 1024: 33). The multiply-adds and the shared-memory reads that feed them bound it (eight
// 16-byte reads per 64 multiply-adds). The gradient of 4 x 8 heads x 2048 x 64, w = 1024: 1.4
// ms, 23 TFLOP/s of 10 d per visible pair (its two kernels form the scores twice: 14 d).
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "sink.cuh"

namespace based {
namespace {

constexpr int T = 64;                        // tile rows
constexpr int kThreads = 256;
constexpr float kLog2e = 1.44269504088896340736f;

template <int D> constexpr int kPitch = D + 4;     // row pitch of a [64][D] tile: float4 rows 4 apart miss each other's banks
constexpr int kPPitch = T + 4;

// Rows [r0, r0 + 64) of a [N, D] slice into shared memory as floats; rows at or
// past `rows` are zero (padding and the sequence's end never reach a product).
template <int D>
__device__ __forceinline__ void load_tile(float* s, const float* g, long long sn, int r0, int rows) {
    for (int i = threadIdx.x; i < T * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = 4 * (i % (D / 4));
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r0 + r < rows) v = load4(g + (r0 + r) * sn + c);
        *reinterpret_cast<float4*>(s + r * kPitch<D> + c) = v;
    }
}

// The same by asynchronous copies (fp32), which land behind the arithmetic on another tile.
template <int D>
__device__ __forceinline__ void copy_tile(float* s, const float* g, long long sn, int r0, int rows) {
    for (int i = threadIdx.x; i < T * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = 4 * (i % (D / 4));
        const bool in = r0 + r < rows;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(s + r * kPitch<D> + c)),
                     "l"(g + (in ? r0 + r : r0) * sn + c), "r"(in ? 16 : 0)
                     : "memory");
    }
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// Two fp32 multiply-adds in one instruction: the same rate, half the issue slots.
using F2 = unsigned long long;
__device__ __forceinline__ F2 pair(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float lo(F2 x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float hi(F2 x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ void fma2(F2& acc, F2 a, F2 b) { asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b)); }
__device__ __forceinline__ ulonglong2 load_pairs(const float* p) { return *reinterpret_cast<const ulonglong2*>(p); }

// acc[i][c] += A[4 ty + i] . B[tx + 16 c] over D channels (both [64][D] tiles); even and
// odd channels in sums of their own.
template <int D>
__device__ __forceinline__ void dot_tile(const float* A, const float* B, int ty, int tx, float acc[4][4]) {
    F2 s[4][4] = {};
#pragma unroll 4
    for (int k = 0; k < D; k += 4) {
        ulonglong2 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = load_pairs(A + (4 * ty + i) * kPitch<D> + k);
#pragma unroll
        for (int c = 0; c < 4; ++c) b[c] = load_pairs(B + (tx + 16 * c) * kPitch<D> + k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                fma2(s[i][c], a[i].x, b[c].x);
                fma2(s[i][c], a[i].y, b[c].y);
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][c] += lo(s[i][c]) + hi(s[i][c]);
}

// acc[i][m] += sum_j P[4 ty + i][j] B[j][cols(m)] (P [64][64], B [64][D]); pair m of a
// thread is columns 4 tx + 64 (m / 2) + 2 (m % 2) and the next.
template <int D>
__device__ __forceinline__ void mul_tile(const float* P, const float* B, int ty, int tx, F2 acc[4][D / 32]) {
#pragma unroll 2
    for (int j = 0; j < T; j += 4) {
        float p[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(P + (4 * ty + i) * kPPitch + j);
            p[i][0] = v.x, p[i][1] = v.y, p[i][2] = v.z, p[i][3] = v.w;
        }
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
            ulonglong2 b[D / 64];
#pragma unroll
            for (int m = 0; m < D / 64; ++m) b[m] = load_pairs(B + (j + jj) * kPitch<D> + 4 * tx + 64 * m);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const F2 pp = pair(p[i][jj], p[i][jj]);
#pragma unroll
                for (int m = 0; m < D / 64; ++m) {
                    fma2(acc[i][2 * m], pp, b[m].x);
                    fma2(acc[i][2 * m + 1], pp, b[m].y);
                }
            }
        }
    }
}

// acc[i][m] += sum_r P[r][4 ty + i] B[r][cols(m)]: the transposed product (dK, dV).
template <int D>
__device__ __forceinline__ void mul_tile_t(const float* P, const float* B, int ty, int tx, F2 acc[4][D / 32]) {
#pragma unroll 4
    for (int r = 0; r < T; ++r) {
        const float4 p = *reinterpret_cast<const float4*>(P + r * kPPitch + 4 * ty);
        const F2 pp[4] = {pair(p.x, p.x), pair(p.y, p.y), pair(p.z, p.z), pair(p.w, p.w)};
#pragma unroll
        for (int m = 0; m < D / 64; ++m) {
            const ulonglong2 b = load_pairs(B + r * kPitch<D> + 4 * tx + 64 * m);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                fma2(acc[i][2 * m], pp[i], b.x);
                fma2(acc[i][2 * m + 1], pp[i], b.y);
            }
        }
    }
}
// Four columns of an accumulator row, times f.
__device__ __forceinline__ float4 quad(const F2* acc, float f) {
    return make_float4(lo(acc[0]) * f, hi(acc[0]) * f, lo(acc[1]) * f, hi(acc[1]) * f);
}

__device__ __forceinline__ float half_warp_max(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float half_warp_sum(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Query block -> (b, h, first row), the longest sweeps first.
struct QBlock {
    int b, h, i0, len;
};
__device__ __forceinline__ QBlock q_block(const SinkArgs& a) {
    const int nt = (a.N + T - 1) / T, bh = a.B * a.Hq;
    QBlock q;
    const int u = blockIdx.x;
    q.i0 = (nt - 1 - u / bh) * T;
    q.b = (u % bh) / a.Hq;
    q.h = (u % bh) % a.Hq;
    q.len = seq_len(a.lengths, q.b, a.N, a.status);
    return q;
}

// The key tiles a query tile at i0 sees: tile 0 for its sinks if the window has left it, then [lo, hi].
struct KeySweep {
    int sink, lo, hi;
    __device__ __forceinline__ KeySweep(const SinkArgs& a, int i0) {
        lo = max(0, i0 - a.w + 1) / T;
        hi = i0 / T;
        sink = (a.n_sink > 0 && lo > 0) ? 1 : 0;
    }
    __device__ __forceinline__ int count() const { return hi - lo + 1 + sink; }
    __device__ __forceinline__ int tile(int s) const { return s < sink ? 0 : lo + s - sink; }
};

// Pairs of K and V tiles in shared memory: at d = 64, where two blocks of an SM still find
// room, the next one is on its way (forward, 4 x 8 heads x 2048 x 64, w = 1024: 423 -> 394
// us); at d = 128 a second would cost a block.
template <int D> constexpr int kRing = D == 64 ? 2 : 1;

// Starts the copy of step s + 1 (of step s where the ring has one pair) and waits for step s.
template <int RING, typename F>
__device__ __forceinline__ void next_pair(int s, int count, F&& fetch) {
    if (RING == 1) fetch(s);
    if (RING > 1 && s + 1 < count) {
        fetch(s + 1);
        copies_wait<1>();
    } else {
        copies_wait<0>();
    }
    __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(kThreads) sink_fwd_kernel(const __grid_constant__ SinkArgs a) {
    extern __shared__ float4 smem4[];
    float* sQ = reinterpret_cast<float*>(smem4);
    float* ring = sQ + T * kPitch<D>;            // K (then the weights P of the same tile) and V
    grid_dependency_wait();
    if (a.fill) grid_launch_dependents();                    // the cache's fill may start
    const QBlock q = q_block(a);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, hk = q.h / (a.Hq / a.Hkv);
    F2 o[4][D / 32] = {};
    float m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = -INFINITY, l[i] = 0.f;
    if (q.i0 < q.len) {
        const float* gq = static_cast<const float*>(a.q.p) + q.b * a.q.sb + q.h * a.q.sh;
        const float* gk = static_cast<const float*>(a.k.p) + q.b * a.k.sb + hk * a.k.sh;
        const float* gv = static_cast<const float*>(a.v.p) + q.b * a.v.sb + hk * a.v.sh;
        load_tile<D>(sQ, gq, a.q.sn, q.i0, q.len);
        const KeySweep ks(a, q.i0);
        const auto fetch = [&](int s) {
            float* at = ring + s % kRing<D> * 2 * T * kPitch<D>;
            copy_tile<D>(at, gk, a.k.sn, ks.tile(s) * T, q.len);
            copy_tile<D>(at + T * kPitch<D>, gv, a.v.sn, ks.tile(s) * T, q.len);
            copies_commit();
        };
        if (kRing<D> > 1) fetch(0);
        for (int s = 0; s < ks.count(); ++s) {
            const int j0 = ks.tile(s) * T;
            float *sK = ring + s % kRing<D> * 2 * T * kPitch<D>, *sV = sK + T * kPitch<D>, *sP = sK;
            next_pair<kRing<D>>(s, ks.count(), fetch);
            float sc[4][4] = {};
            dot_tile<D>(sQ, sK, ty, tx, sc);
            __syncthreads();                     // sK is read; P takes its place
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = q.i0 + 4 * ty + i;
                float mx = -INFINITY;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int j = j0 + tx + 16 * c;
                    sc[i][c] = visible(row, j, a.w, a.n_sink) ? sc[i][c] * a.scale : -INFINITY;
                    mx = fmaxf(mx, sc[i][c]);
                }
                const float mn = fmaxf(m[i], half_warp_max(mx));
                const float mu = mn == -INFINITY ? 0.f : mn;             // nothing seen yet
                const float al = expf(m[i] - mu);
                float sum = 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float p = expf(sc[i][c] - mu);
                    sum += p;
                    sP[(4 * ty + i) * kPPitch + tx + 16 * c] = p;
                }
                l[i] = l[i] * al + half_warp_sum(sum);
                m[i] = mn;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) o[i][c] = pair(lo(o[i][c]) * al, hi(o[i][c]) * al);
            }
            __syncthreads();
            mul_tile<D>(sP, sV, ty, tx, o);
            __syncthreads();
        }
    }
    float* gy = static_cast<float*>(a.y.p) + q.b * a.y.sb + q.h * a.y.sh;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = q.i0 + 4 * ty + i;
        if (row >= a.N) continue;
        const bool pad = row >= q.len;
        const float inv = pad ? 0.f : 1.0f / l[i];
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            float4 v = quad(o[i] + 2 * c, inv);
            if (pad) v = make_float4(0.f, 0.f, 0.f, 0.f);
            store4(gy + row * a.y.sn + 4 * tx + 64 * c, v);
        }
        if (a.lse != nullptr && tx == 0)
            a.lse[((size_t)q.b * a.Hq + q.h) * a.N + row] = pad ? -INFINITY : m[i] + logf(l[i]);
    }
    // Rows that came out non-finite, again from their definition.
    float odd = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < D / 32; ++c) odd = fmaf(lo(o[i][c]), 0.f, fmaf(hi(o[i][c]), 0.f, odd));
    if (!__syncthreads_or(odd != 0.f)) return;
    const KeySweep ks(a, q.i0);
    redo_rows<float, D>(a, q.b, q.h, hk, q.i0, T, q.len, ks.lo * T, ks.sink * T, threadIdx.x >> 5, kThreads / 32);
}

// dQ, and delta_i = dy_i . y_i into the workspace [B, Hq, N].
template <int D>
__global__ void __launch_bounds__(kThreads) sink_dq_kernel(const __grid_constant__ SinkArgs a, float* delta) {
    extern __shared__ float4 smem4[];
    float* sQ = reinterpret_cast<float*>(smem4);
    float* sG = sQ + T * kPitch<D>;              // dy
    float* ring = sG + T * kPitch<D>;            // K and V, then dS of the same tile over V
    grid_dependency_wait();
    const QBlock q = q_block(a);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, hk = q.h / (a.Hq / a.Hkv);
    F2 o[4][D / 32] = {};
    if (q.i0 < q.len) {
        const float* gq = static_cast<const float*>(a.q.p) + q.b * a.q.sb + q.h * a.q.sh;
        const float* gg = static_cast<const float*>(a.dy.p) + q.b * a.dy.sb + q.h * a.dy.sh;
        const float* gk = static_cast<const float*>(a.k.p) + q.b * a.k.sb + hk * a.k.sh;
        const float* gv = static_cast<const float*>(a.v.p) + q.b * a.v.sb + hk * a.v.sh;
        const float* gy = static_cast<const float*>(a.y.p) + q.b * a.y.sb + q.h * a.y.sh;
        load_tile<D>(sQ, gq, a.q.sn, q.i0, q.len);
        load_tile<D>(sG, gg, a.dy.sn, q.i0, q.len);
        load_tile<D>(ring, gy, a.y.sn, q.i0, q.len);
        __syncthreads();
        float dl[4], ls[4];
        const size_t row0 = ((size_t)q.b * a.Hq + q.h) * a.N;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * ty + i, row = q.i0 + r;
            float s = 0.f;
            for (int c = tx; c < D; c += 16) s = fmaf(sG[r * kPitch<D> + c], ring[r * kPitch<D> + c], s);
            dl[i] = half_warp_sum(s);
            ls[i] = row < q.len ? a.lse[row0 + row] : 0.f;
            if (tx == 0 && row < q.len) delta[row0 + row] = dl[i];
        }
        __syncthreads();
        const KeySweep ks(a, q.i0);
        const auto fetch = [&](int s) {
            float* at = ring + s % kRing<D> * 2 * T * kPitch<D>;
            copy_tile<D>(at, gk, a.k.sn, ks.tile(s) * T, q.len);
            copy_tile<D>(at + T * kPitch<D>, gv, a.v.sn, ks.tile(s) * T, q.len);
            copies_commit();
        };
        if (kRing<D> > 1) fetch(0);
        for (int s = 0; s < ks.count(); ++s) {
            const int j0 = ks.tile(s) * T;
            float *sK = ring + s % kRing<D> * 2 * T * kPitch<D>, *sV = sK + T * kPitch<D>, *sS = sV;
            next_pair<kRing<D>>(s, ks.count(), fetch);
            float sc[4][4] = {}, dp[4][4] = {};
            dot_tile<D>(sQ, sK, ty, tx, sc);
            dot_tile<D>(sG, sV, ty, tx, dp);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = q.i0 + 4 * ty + i;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const bool see = row < q.len && visible(row, j0 + tx + 16 * c, a.w, a.n_sink);
                    const float p = expf(sc[i][c] * a.scale - ls[i]);
                    sS[(4 * ty + i) * kPPitch + tx + 16 * c] = see ? a.scale * p * (dp[i][c] - dl[i]) : 0.f;
                }
            }
            __syncthreads();
            mul_tile<D>(sS, sK, ty, tx, o);
            __syncthreads();
        }
    }
    float* out = static_cast<float*>(a.dq.p) + q.b * a.dq.sb + q.h * a.dq.sh;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);     // padding rows: 0 times an infinite key is not
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = q.i0 + 4 * ty + i;
        if (row >= a.N) continue;
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
            store4(out + row * a.dq.sn + 4 * tx + 64 * c, row < q.len ? quad(o[i] + 2 * c, 1.0f) : zero);
    }
    // Rows that came out non-finite, again from their definition.
    float odd = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < D / 32; ++c) odd = fmaf(lo(o[i][c]), 0.f, fmaf(hi(o[i][c]), 0.f, odd));
    if (!__syncthreads_or(odd != 0.f)) return;
    const size_t row0 = ((size_t)q.b * a.Hq + q.h) * a.N;
    bool checked = false;
    for (int row = q.i0 + (threadIdx.x >> 5); row < min(q.i0 + T, q.len); row += kThreads / 32) {
        float* at = row_of<float>(a.dq, q.b, q.h, row);
        if (!odd_row<D>(at)) continue;
        const KeySweep ks(a, q.i0);
        if (!checked && !odd_hidden_keys<D>(row_of<const float>(a.k, q.b, hk, 0), a.k.sn, q.i0, T, q.len, ks.lo * T, a.w,
                                            a.n_sink, ks.sink * T))
            break;
        checked = true;
        const GradRow<D> x =
            sink_exact_dq<float, D>(a, q.b, q.h, hk, row, a.scale * kLog2e, a.lse + row0, -kLog2e, delta + row0);
        put_row<D>(at, x.a, a.scale);
    }
}

// dK, dV of one unit (see SinkSplit in sink.cuh).
template <int D>
__global__ void __launch_bounds__(kThreads) sink_dkv_kernel(const __grid_constant__ SinkArgs a, SinkSplit sp,
                                                            FastDiv by_bh, FastDiv by_h,
                                                            const float* delta, float* partial) {
    extern __shared__ float4 smem4[];
    float* sK = reinterpret_cast<float*>(smem4);
    float* sV = sK + T * kPitch<D>;
    float* sQ = sV + T * kPitch<D>;
    float* sG = sQ + T * kPitch<D>;
    float* sP = sG + T * kPitch<D>;
    float* sS = sP + T * kPPitch;
    grid_dependency_wait();
    const SinkUnit u = sink_unit(sp, blockIdx.x, by_bh, by_h);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int len = seq_len(a.lengths, u.b, a.N, a.status);
    const int j0 = u.kt * T, group = a.Hq / a.Hkv;
    F2 dk[4][D / 32] = {}, dv[4][D / 32] = {};
    if (j0 < len) {
        const float* gk = static_cast<const float*>(a.k.p) + u.b * a.k.sb + u.hk * a.k.sh;
        const float* gv = static_cast<const float*>(a.v.p) + u.b * a.v.sb + u.hk * a.v.sh;
        load_tile<D>(sK, gk, a.k.sn, j0, len);
        load_tile<D>(sV, gv, a.v.sn, j0, len);
        for (int s = u.s0; s < u.s1; ++s) {
            const int h = u.hk * group + s / u.span, i0 = (u.t0 + s % u.span) * T;
            if (i0 >= len) continue;
            const float* gq = static_cast<const float*>(a.q.p) + u.b * a.q.sb + h * a.q.sh;
            const float* gg = static_cast<const float*>(a.dy.p) + u.b * a.dy.sb + h * a.dy.sh;
            __syncthreads();
            copy_tile<D>(sQ, gq, a.q.sn, i0, len);
            copy_tile<D>(sG, gg, a.dy.sn, i0, len);
            copies_commit();
            copies_wait<0>();
            __syncthreads();
            float sc[4][4] = {}, dp[4][4] = {};
            dot_tile<D>(sQ, sK, ty, tx, sc);
            dot_tile<D>(sG, sV, ty, tx, dp);
            const size_t row0 = ((size_t)u.b * a.Hq + h) * a.N;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = i0 + 4 * ty + i;
                const float ls = row < len ? a.lse[row0 + row] : 0.f, dl = row < len ? delta[row0 + row] : 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int j = j0 + tx + 16 * c;
                    const bool see = row < len && j <= row &&
                                     (u.chunk < 0 ? j > row - a.w : (j < a.n_sink && j <= row - a.w));
                    const float p = see ? expf(sc[i][c] * a.scale - ls) : 0.f;
                    sP[(4 * ty + i) * kPPitch + tx + 16 * c] = p;
                    sS[(4 * ty + i) * kPPitch + tx + 16 * c] = see ? a.scale * p * (dp[i][c] - dl) : 0.f;
                }
            }
            __syncthreads();
            mul_tile_t<D>(sP, sG, ty, tx, dv);
            mul_tile_t<D>(sS, sQ, ty, tx, dk);
        }
    }
    float* ok = static_cast<float*>(a.dk.p) + u.b * a.dk.sb + u.hk * a.dk.sh;
    float* ov = static_cast<float*>(a.dv.p) + u.b * a.dv.sb + u.hk * a.dv.sh;
    // Partials go to slot 0 (the sink tile's band unit) or 1 + chunk: rows of the sinks only.
    float* part = partial + sink_partial_offset(sp, u.b * a.Hkv + u.hk, u.chunk + 1, D);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i, row = j0 + r;
        if (row >= a.N) continue;
        const bool sink = sp.chunks > 0 && row < a.n_sink;
        if (u.chunk >= 0 && !sink) continue;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            float4 fk = quad(dk[i] + 2 * c, 1.0f), fv = quad(dv[i] + 2 * c, 1.0f);
            if (row >= len) fk = fv = make_float4(0.f, 0.f, 0.f, 0.f);
            const int col = 4 * tx + 64 * c;
            if (sink) {
                store4(part + r * D + col, fk);
                store4(part + (sp.rows + r) * D + col, fv);
            } else {
                store4(ok + row * a.dk.sn + col, fk);
                store4(ov + row * a.dv.sn + col, fv);
            }
        }
    }
    // Rows that came out non-finite, again from their definition.
    float odd = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
            odd = fmaf(lo(dk[i][c]), 0.f, fmaf(hi(dk[i][c]), 0.f, fmaf(lo(dv[i][c]), 0.f, fmaf(hi(dv[i][c]), 0.f, odd))));
    if (!__syncthreads_or(odd != 0.f)) return;
    bool checked = false;
    for (int j = j0 + (threadIdx.x >> 5); j < min(j0 + T, len); j += kThreads / 32) {
        const bool sink = sp.chunks > 0 && j < a.n_sink;     // a row of the unit's partials
        if (u.chunk >= 0 && !sink) break;
        float* pk = sink ? part + (size_t)(j - j0) * D : row_of<float>(a.dk, u.b, u.hk, j);
        float* pv = sink ? pk + (size_t)sp.rows * D : row_of<float>(a.dv, u.b, u.hk, j);
        if (!odd_row<D>(pk) && !odd_row<D>(pv)) continue;
        if (!checked && !odd_hidden_queries<D, float>(a, u.b, u.hk * group, group, u.chunk >= 0, j0, T, len, u.t0 * T,
                                                      (u.t0 + u.span) * T))
            break;
        checked = true;
        GradRow<D> x;
        for (int s = u.s0; s < u.s1; ++s) {
            const int i0 = (u.t0 + s % u.span) * T;
            const int from = u.chunk < 0 ? j : j + a.w, end = u.chunk < 0 ? min(len, j + a.w) : len;
            sink_exact_dkv<float, D>(x, a, u.b, u.hk * group + s / u.span, u.hk, j, max(i0, from), min(i0 + T, end),
                                     a.scale * kLog2e, a.lse, -kLog2e, delta, a.N);
        }
        put_row<D>(pk, x.a, a.scale);
        put_row<D>(pv, x.b, 1.0f);
    }
}

template <int D>
cudaError_t prefill(const SinkArgs& a, cudaStream_t stream) {
    constexpr int smem = (1 + 2 * kRing<D>) * T * kPitch<D> * 4;
    auto kern = sink_fwd_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((unsigned)(a.B * a.Hq * ((a.N + T - 1) / T))), dim3(kThreads), smem, stream, a);
}

template <int D>
cudaError_t backward(const SinkArgs& a, cudaStream_t stream) {
    constexpr int smem_q = (2 + 2 * kRing<D>) * T * kPitch<D> * 4, smem_k = (4 * kPitch<D> + 2 * kPPitch) * T * 4;
    auto kq = sink_dq_kernel<D>;
    auto kk = sink_dkv_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(kq, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_q);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kk, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_k);
    if (e != cudaSuccess) return e;
    const SinkSplit sp = sink_split(a.Hq, a.Hkv, a.N, a.w, a.n_sink, T, T);
    float* delta = static_cast<float*>(a.workspace);
    float* partial = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + sink_delta_bytes(a.B, a.Hq, a.N));
    e = launch_pdl(kq, dim3((unsigned)(a.B * a.Hq * ((a.N + T - 1) / T))), dim3(kThreads), smem_q, stream, a, delta);
    if (e == cudaSuccess)
        e = launch_pdl(kk, dim3((unsigned)(a.B * a.Hkv * sp.units())), dim3(kThreads), smem_k, stream, a, sp,
                       FastDiv(a.B * a.Hkv), FastDiv(a.Hkv), static_cast<const float*>(delta), partial);
    if (e == cudaSuccess && sp.chunks > 0) e = launch_sink_join<float>(a, sp, partial, stream);
    return e;
}

template <typename E>
__global__ void __launch_bounds__(256) sink_join_kernel(const __grid_constant__ SinkArgs a, SinkSplit sp,
                                                        const float* partial) {
    grid_dependency_wait();
    const int per = a.n_sink * a.d / 4, total = 2 * per;
    const int bh = blockIdx.x, b = bh / a.Hkv, hk = bh % a.Hkv;
    for (int i = blockIdx.y * 256 + threadIdx.x; i < total; i += gridDim.y * 256) {
        const int which = i / per, r = (i % per) * 4 / a.d, c = (i % per) * 4 % a.d;
        if (r >= a.N) continue;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k <= sp.chunks; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(partial + sink_partial_offset(sp, bh, k, a.d) +
                                                              (size_t)(which * sp.rows + r) * a.d + c);
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        const View& o = which == 0 ? a.dk : a.dv;
        store4(static_cast<E*>(o.p) + b * o.sb + hk * o.sh + r * o.sn + c, s);
    }
}

// 16-byte pieces of the cache: slot t < n_sink holds token t, slot n_sink + r the
// latest token t >= n_sink with (t - n_sink) mod w = r; the others are zero.
// It needs nothing of the attention before it in the stream, but k and v may come from the
// kernel before that, whose writes are visible only behind the wait. Its blocks are in place by
// then: only before it do the attention's kernels let their successor start early (another of
// their own, with blocks that stay, would be spread unevenly over the SMs: 37 -> 42 us).
__global__ void __launch_bounds__(256) sink_cache_kernel(const __grid_constant__ SinkArgs a, uint4* kc, uint4* vc,
                                                         int esize) {
    grid_dependency_wait();
    const int slots = a.n_sink + a.w, pieces = a.d * esize / 16;
    const int b = blockIdx.x / a.Hkv, hk = blockIdx.x % a.Hkv;
    const int len = seq_len(a.lengths, b, a.N, a.status);
    const size_t base = ((size_t)b * a.Hkv + hk) * slots;
    const char* gk = static_cast<const char*>(a.k.p) + (b * a.k.sb + hk * a.k.sh) * esize;
    const char* gv = static_cast<const char*>(a.v.p) + (b * a.v.sb + hk * a.v.sh) * esize;
    for (long long i = (long long)blockIdx.y * 256 + threadIdx.x; i < (long long)slots * pieces;
         i += (long long)gridDim.y * 256) {
        const int slot = (int)(i / pieces), piece = (int)(i % pieces);
        int tok = slot;
        if (slot >= a.n_sink) {
            const int last = len - 1 - slot;             // len - 1 - n_sink - r
            tok = last >= 0 ? slot + last / a.w * a.w : -1;
        } else if (slot >= len) {
            tok = -1;
        }
        uint4 x = make_uint4(0, 0, 0, 0), y = x;
        if (tok >= 0) {
            x = *reinterpret_cast<const uint4*>(gk + tok * a.k.sn * esize + 16 * piece);
            y = *reinterpret_cast<const uint4*>(gv + tok * a.v.sn * esize + 16 * piece);
        }
        kc[(base + slot) * pieces + piece] = x;
        vc[(base + slot) * pieces + piece] = y;
    }
}

}  // namespace

template <typename E>
cudaError_t launch_sink_join(const SinkArgs& a, const SinkSplit& sp, const float* partial, cudaStream_t stream) {
    const int blocks = (2 * a.n_sink * a.d / 4 + 255) / 256;
    return launch_pdl(sink_join_kernel<E>, dim3(a.B * a.Hkv, blocks), dim3(256), 0, stream, a, sp, partial);
}
template cudaError_t launch_sink_join<float>(const SinkArgs&, const SinkSplit&, const float*, cudaStream_t);
template cudaError_t launch_sink_join<__nv_bfloat16>(const SinkArgs&, const SinkSplit&, const float*, cudaStream_t);

cudaError_t launch_sink_prefill_f32(const SinkArgs& a, cudaStream_t stream) {
    return a.d == 64 ? prefill<64>(a, stream) : prefill<128>(a, stream);
}

cudaError_t launch_sink_backward_f32(const SinkArgs& a, cudaStream_t stream) {
    return a.d == 64 ? backward<64>(a, stream) : backward<128>(a, stream);
}

size_t sink_backward_workspace(int B, int Hq, int Hkv, int N, int d, int w, int n_sink, bool bf16) {
    if (bf16) return sink_backward_workspace_tc(B, Hq, Hkv, N, d, w, n_sink);
    const SinkSplit sp = sink_split(Hq, Hkv, N, w, n_sink, T, T);
    return sink_delta_bytes(B, Hq, N) + sink_partial_offset(sp, B * Hkv, 0, d) * sizeof(float);
}

cudaError_t launch_sink_cache_fill(const SinkArgs& a, void* k_cache, void* v_cache, bool bf16, cudaStream_t stream) {
    const int esize = bf16 ? 2 : 4;
    const long long pieces = (long long)(a.n_sink + a.w) * (a.d * esize / 16);
    const unsigned by = (unsigned)std::min<long long>((pieces + 255) / 256, 1024);
    return launch_pdl(sink_cache_kernel, dim3(a.B * a.Hkv, by), dim3(256), 0, stream, a,
                      static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), esize);
}

}  // namespace based
