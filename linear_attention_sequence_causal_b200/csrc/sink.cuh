// Shared by the kernels of the sliding-window attention with sink tokens.
#pragma once

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace based {

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// s + the dot product of two 16-byte pieces (the last argument gives the type).
__device__ __forceinline__ float dot16(uint4 a, uint4 b, float s, const float*) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fmaf(__uint_as_float(x[i]), __uint_as_float(y[i]), s);
    return s;
}
__device__ __forceinline__ float dot16(uint4 a, uint4 b, float s, const __nv_bfloat16*) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), s);
        s = fmaf(__uint_as_float(x[i] & 0xFFFF0000u), __uint_as_float(y[i] & 0xFFFF0000u), s);
    }
    return s;
}

// The dot product of two rows, the loads of four pieces in flight.
template <typename E, int D>
__device__ __forceinline__ float dot_row(const E* q, const E* k) {
    constexpr int P = 16 / (int)sizeof(E);                   // channels of a 16-byte piece
    float s = 0.f;
#pragma unroll 1
    for (int c = 0; c < D; c += 4 * P) {
        uint4 a[4], b[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            a[x] = *reinterpret_cast<const uint4*>(q + c + x * P);
            b[x] = *reinterpret_cast<const uint4*>(k + c + x * P);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) s = dot16(a[x], b[x], s, q);
    }
    return s;
}

// One row of the attention from its definition, by a whole warp: lane t gets channels
// t D/32 .. of the output (in .x, .y, ..), all lanes the row's lse. The tiled kernels take
// it for rows that come out non-finite: there a weight of 0 may have met an infinity or a
// NaN in the values of a token that shares the tile but that the row does not see.
// 32 keys at a time, a key per lane: tens of cycles per key. The tensor-core kernels take such
// rows once their roles are through, so that no bounded wait runs out over them. A NaN among
// the scores makes the whole row NaN and ends it.
template <typename E, int D>
__device__ __noinline__ float4 sink_exact_row(const E* q, const E* k, const E* v, long long k_sn, long long v_sn, int i,
                                              int w, int n_sink, float scale, float* lse) {
    constexpr int CH = D / 32;
    const int lane = threadIdx.x & 31, c0 = lane * CH;
    float acc[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) acc[c] = 0.f;
    float m = -INFINITY, l = 0.f;
    const int lo = max(0, i - w + 1), sinks = min(n_sink, lo), total = sinks + i + 1 - lo;
    for (int t0 = 0; t0 < total && l == l; t0 += 32) {       // t: the sinks below the window, then the window
        const int t = t0 + lane;
        float s = -INFINITY;
        if (t < total) {
            const E* kr = k + (long long)(t < sinks ? t : lo + t - sinks) * k_sn;
            s = dot_row<E, D>(q, kr) * scale;
        }
        float mx = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mn = fmaxf(m, mx), mu = mn == -INFINITY ? 0.f : mn;
        const float f = expf(m - mu), p = expf(s - mu);
        float sum = p;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l = l * f + sum;
        m = mn;
#pragma unroll
        for (int c = 0; c < CH; ++c) acc[c] *= f;
        const int n = min(32, total - t0);
        for (int j0 = 0; j0 < n; j0 += 8) {                  // the loads of eight rows in flight
            E x[8][CH];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int tj = min(t0 + j0 + u, total - 1);
                const E* vr = v + (long long)(tj < sinks ? tj : lo + tj - sinks) * v_sn + c0;
#pragma unroll
                for (int c = 0; c < CH; ++c) x[u][c] = vr[c];
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float pj = __shfl_sync(0xffffffffu, p, j0 + u);
                if (j0 + u < n) {
#pragma unroll
                    for (int c = 0; c < CH; ++c) acc[c] = fmaf(pj, to_f32(x[u][c]), acc[c]);
                }
            }
        }
    }
    *lse = m + logf(l);
    const float inv = 1.0f / l;
    return make_float4(acc[0] * inv, acc[1] * inv, CH > 2 ? acc[CH - 2] * inv : 0.f, CH > 2 ? acc[CH - 1] * inv : 0.f);
}

// A row of the gradient from its definition, for the same reason: a hidden pair's weight of 0
// may have met an infinity or a NaN. Lane t holds channels t D/32 ..
template <int D>
struct GradRow {
    float a[D / 32], b[D / 32];              // DQ: dq, unused; DKV: dk, dv (without the factor `scale`)
    __device__ __forceinline__ GradRow() {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) a[c] = b[c] = 0.f;
    }
    // Whether every channel is NaN, which no further term changes.
    __device__ __forceinline__ bool lost(bool both) const {
        bool nan = true;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) nan = nan && a[c] != a[c] && (!both || b[c] != b[c]);
        return __all_sync(0xffffffffu, nan);
    }
};

// Adds the terms of the keys (DQ) or queries (DKV) [from, to) to `acc`, by a whole warp.
// x0, x1: the row's q and dy with a, b the keys and values, or its k and v with a, b the
// queries and their dy. With m lse + c s the exponent of p and delta = dy . y, both by query:
// ds = p (x1 . b - delta), acc.a += ds a, acc.b += p b. i: the query of DQ.
template <typename E, int D, bool DKV>
__device__ __forceinline__ void sink_exact_terms(GradRow<D>& acc, const E* x0, const E* x1, const E* a, long long a_sn,
                                                 const E* b, long long b_sn, int from, int to, float c, const float* lse,
                                                 float m, const float* delta, int i) {
    constexpr int CH = D / 32;
    const int lane = threadIdx.x & 31, c0 = lane * CH;
    for (int t0 = from; t0 < to && !acc.lost(DKV); t0 += 32) {
        const int t = t0 + lane;
        float p = 0.f, ds = 0.f;
        if (t < to) {
            const int at = DKV ? t : i;
            p = exp2f(fmaf(dot_row<E, D>(x0, a + t * a_sn), c, m * lse[at]));
            ds = p * (dot_row<E, D>(x1, b + t * b_sn) - delta[at]);
        }
        const int n = min(32, to - t0);
        for (int j0 = 0; j0 < n; j0 += 4) {                  // the loads of four rows in flight
            E x[4][CH], z[4][CH];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const long long tj = min(t0 + j0 + u, to - 1);
#pragma unroll
                for (int e = 0; e < CH; ++e) {
                    x[u][e] = a[tj * a_sn + c0 + e];
                    if (DKV) z[u][e] = b[tj * b_sn + c0 + e];
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float dj = __shfl_sync(0xffffffffu, ds, j0 + u), pj = __shfl_sync(0xffffffffu, p, j0 + u);
                if (j0 + u < n) {
#pragma unroll
                    for (int e = 0; e < CH; ++e) {
                        acc.a[e] = fmaf(dj, to_f32(x[u][e]), acc.a[e]);
                        if (DKV) acc.b[e] = fmaf(pj, to_f32(z[u][e]), acc.b[e]);
                    }
                }
            }
        }
    }
}

// Row h, n of batch b of a view.
template <typename E>
__device__ __forceinline__ E* row_of(const View& v, int b, int h, int n) {
    return static_cast<E*>(v.p) + b * v.sb + h * v.sh + n * v.sn;
}

// dq of query i without the factor `scale`; lse and delta of the head's queries.
template <typename E, int D, typename P>
__device__ __forceinline__ GradRow<D> sink_exact_dq(const P& p, int b, int h, int hk, int i, float c, const float* lse, float m,
                                                    const float* delta) {
    GradRow<D> acc;
    const int lo = max(0, i - p.w + 1);
#pragma unroll 1
    for (int part = 0; part < 2; ++part)                     // the sinks below the window, the window
        sink_exact_terms<E, D, false>(acc, row_of<const E>(p.q, b, h, i), row_of<const E>(p.dy, b, h, i),
                                      row_of<const E>(p.k, b, hk, 0), p.k.sn, row_of<const E>(p.v, b, hk, 0), p.v.sn,
                                      part ? lo : 0, part ? i + 1 : min(p.n_sink, lo), c, lse, m, delta, i);
    return acc;
}

// Adds the queries [from, to) of head h to dk, dv of key j; lse and delta of head 0 of batch
// 0, `pitch` floats per head.
template <typename E, int D, typename P>
__device__ __forceinline__ void sink_exact_dkv(GradRow<D>& acc, const P& p, int b, int h, int hk, int j, int from, int to,
                                               float c, const float* lse, float m, const float* delta, int pitch) {
    const size_t at = ((size_t)b * p.Hq + h) * pitch;
    sink_exact_terms<E, D, true>(acc, row_of<const E>(p.k, b, hk, j), row_of<const E>(p.v, b, hk, j),
                                 row_of<const E>(p.q, b, h, 0), p.q.sn, row_of<const E>(p.dy, b, h, 0), p.dy.sn, from, to, c,
                                 lse + at, m, delta + at, 0);
}

// Whether one of this lane's channels of a row is not finite; of a row; of the rows [r0, r1).
template <int D>
__device__ __forceinline__ bool odd_channels(const __nv_bfloat16* row) {
    bool odd = false;                                        // an exponent of all ones
#pragma unroll
    for (int c = 0; c < D / 32; c += 2) {
        const uint32_t x = __ldcg(reinterpret_cast<const uint32_t*>(row + (threadIdx.x & 31) * (D / 32) + c));
        odd |= (x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u;
    }
    return odd;
}
template <int D>
__device__ __forceinline__ bool odd_channels(const float* row) {
    float odd = 0.f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) odd = fmaf(__ldcg(row + (threadIdx.x & 31) * (D / 32) + c), 0.f, odd);
    return odd != 0.f;
}
template <int D, typename E>
__device__ __forceinline__ bool odd_row(const E* row) {
    return __any_sync(0xffffffffu, odd_channels<D>(row));
}
template <int D, typename E>
__device__ __forceinline__ bool odd_rows(const E* x, long long sn, int r0, int r1) {
    bool odd = false;
#pragma unroll 8
    for (int r = r0; r < r1; ++r) odd |= odd_channels<D>(x + r * sn);
    return __any_sync(0xffffffffu, odd);
}
// Whether the keys [first, ..) that the products of the query rows [i0, i0 + rows) took hold a
// non-finite value hidden from one of them: below the last row's window, or behind the first
// row; or a sink block of sink_rows keys, behind the sinks. Where they do not, non-finite
// results are the definition's own and stay.
template <int D, typename E>
__device__ __forceinline__ bool odd_hidden_keys(const E* x, long long sn, int i0, int rows, int len, int first, int w,
                                                int n_sink, int sink_rows) {
    return odd_rows<D>(x, sn, max(first, n_sink), min(i0 + rows - w, len)) || odd_rows<D>(x, sn, i0 + 1, min(i0 + rows, len)) ||
           odd_rows<D>(x, sn, n_sink, sink_rows);
}
// The same for the queries up to `last` of the group's heads h .. that the products of the
// keys [j0, j0 + rows) took (chunk: of the sinks, from query `first` on).
template <int D, typename E, typename P>
__device__ __forceinline__ bool odd_hidden_queries(const P& p, int b, int h, int heads, bool chunk, int j0, int rows, int len,
                                                   int first, int last) {
    bool odd = false;
#pragma unroll 1
    for (int x = 0; x < 2 * heads && !odd; ++x) {
        const View& v = x & 1 ? p.dy : p.q;
        const E* at = row_of<const E>(v, b, h + (x >> 1), 0);
        odd = odd_rows<D>(at, v.sn, chunk ? first : j0, min(len, chunk ? p.n_sink + p.w : j0 + rows)) ||
              (!chunk && odd_rows<D>(at, v.sn, j0 + p.w, min(len, last)));
    }
    return odd;
}
template <int D, typename E>
__device__ __forceinline__ void put_row(E* row, const float* x, float f) {
#pragma unroll
    for (int c = 0; c < D / 32; ++c) row[(threadIdx.x & 31) * (D / 32) + c] = from_f32<E>(x[c] * f);
}

// Rows i0 + warp, i0 + warp + warps, .. of a query tile of a finished block, each by a whole
// warp: y and lse computed again from their definition (see sink_exact_row) where they came
// out non-finite and a hidden value of the key tiles from `first` on may be why. P: q, k, v, ..
template <typename E, int D, typename P>
__device__ __forceinline__ void redo_rows(const P& p, int b, int h, int hk, int i0, int rows, int len, int first,
                                          int sink_rows, int warp, int warps) {
    bool checked = false;
    for (int i = i0 + warp; i < min(i0 + rows, len); i += warps) {
        E* y = row_of<E>(p.y, b, h, i);
        if (!odd_row<D>(y)) continue;
        if (!checked && !odd_hidden_keys<D>(row_of<const E>(p.v, b, hk, 0), p.v.sn, i0, rows, len, first, p.w, p.n_sink,
                                            sink_rows))
            return;
        checked = true;
        float ls;
        const float4 x = sink_exact_row<E, D>(row_of<const E>(p.q, b, h, i), row_of<const E>(p.k, b, hk, 0),
                                               row_of<const E>(p.v, b, hk, 0), p.k.sn, p.v.sn, i, p.w, p.n_sink, p.scale, &ls);
        const float xs[4] = {x.x, x.y, x.z, x.w};
        put_row<D>(y, xs, 1.0f);
        if (p.lse != nullptr && (threadIdx.x & 31) == 0) p.lse[((size_t)b * p.Hq + h) * p.N + i] = ls;
    }
}

// Division of a non-negative 31-bit number by a constant of the launch: multiply and
// shift in place of the ~150 cycles that a division by a variable takes, which every
// role of a persistent block would spend several of per unit.
struct FastDiv {
    uint32_t d, mul, shift;
    FastDiv() = default;
    explicit FastDiv(int divisor) : d((uint32_t)divisor), mul(0), shift(0) {
        while ((1ull << shift) < d) ++shift;                 // 2^shift >= d
        mul = (uint32_t)(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
    }
    // floor(n / d): the high word of n (2^32 + mul) / 2^32, whose error stays below 1 / d for n < 2^31.
    __host__ __device__ inline int div(int n) const {
#ifdef __CUDA_ARCH__
        const uint32_t high = __umulhi((uint32_t)n, mul);
#else
        const uint32_t high = (uint32_t)(((uint64_t)(uint32_t)n * mul) >> 32);
#endif
        return (int)((high + (uint32_t)n) >> shift);
    }
    __host__ __device__ inline int mod(int n) const { return n - div(n) * (int)d; }
};

// A row of bf16 outputs, 16 channels at a time: one 32-byte store where the rows allow
// it (a whole sector; the 16-byte ones write half sectors and take twice the store
// unit's time, which shows at the end of short units), else two of 16.
__device__ __forceinline__ void store16(__nv_bfloat16* p, uint4 a, uint4 b, bool aligned32) {
    if (aligned32) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
                     "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = a;
        reinterpret_cast<uint4*>(p)[1] = b;
    }
}
// Whether every row of a bf16 view starts on a 32-byte boundary.
inline bool rows_aligned32(const View& v) {
    return (reinterpret_cast<uintptr_t>(v.p) & 31) == 0 && (v.sb | v.sh | v.sn) % 16 == 0;
}

// Tokens of sequence b, clamped to [0, N]; a value outside is reported.
__device__ __forceinline__ int seq_len(const int64_t* lengths, int b, int N, unsigned* status) {
    if (lengths == nullptr) return N;
    const int64_t n = lengths[b];
    if (n >= 0 && n <= N) return (int)n;
    atomicOr(status, DEV_ERR_RANGE);
    return n < 0 ? 0 : N;
}

__device__ __forceinline__ bool visible(int i, int j, int w, int n_sink) {
    return j <= i && (j > i - w || j < n_sink);
}

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// How the dK, dV work of one key/value head is cut into units, for key tiles of T and
// query tiles of TQ rows: nt band units (key tile kt against the query tiles that see it
// through the window, over the group's heads) and `chunks` units of the sink tile, each
// a stretch of `chunk_len` steps of the list (head of the group, query tile past the
// window). A chunk is as long as a full band unit, so the units stay even.
struct SinkSplit {
    int nt, ntq, ratio, chunks, chunk_len, span, t_first, band, group;   // ratio: T / TQ
    int rows;                                // rows of a partial: the sink tokens
    __host__ __device__ int units() const { return nt + chunks; }
};

inline SinkSplit sink_split(int Hq, int Hkv, int N, int w, int n_sink, int T, int TQ) {
    SinkSplit s{};
    s.nt = (N + T - 1) / T;
    s.ntq = (N + TQ - 1) / TQ;
    s.ratio = T / TQ;
    s.group = Hq / Hkv;
    s.rows = n_sink;
    s.band = (int)std::min<long long>(s.ntq, ((long long)T + w - 2) / TQ + 1);
    if (n_sink > 0 && w < N) {               // a query i >= w has sinks outside its window
        s.t_first = w / TQ;
        s.span = s.ntq - s.t_first;
        const long long steps = (long long)s.span * s.group;
        s.chunk_len = std::max(s.band * s.group, 1);
        s.chunks = (int)((steps + s.chunk_len - 1) / s.chunk_len);
    }
    return s;
}

struct SinkUnit {
    int b, hk, kt, chunk;                    // chunk -1: a band unit
    int t0, span, s0, s1;                    // steps [s0, s1): head s / span of the group, query tile t0 + s % span
};

// Unit u of B * Hkv * units(): chunks of the sink tile first, then band units, all
// heads of one kind side by side.
__host__ __device__ inline SinkUnit sink_unit(const SinkSplit& sp, int u, FastDiv by_bh, FastDiv by_h) {
    SinkUnit r;
    const int i = by_bh.div(u), bh = u - i * (int)by_bh.d;
    r.b = by_h.div(bh);
    r.hk = bh - r.b * (int)by_h.d;
    if (i < sp.chunks) {
        r.kt = 0;
        r.chunk = i;
        r.t0 = sp.t_first;
        r.span = sp.span;
        r.s0 = i * sp.chunk_len;
        const int end = sp.span * sp.group;
        r.s1 = r.s0 + sp.chunk_len < end ? r.s0 + sp.chunk_len : end;
    } else {
        r.kt = i - sp.chunks;
        r.chunk = -1;
        r.t0 = r.kt * sp.ratio;
        r.span = r.t0 + sp.band <= sp.ntq ? sp.band : sp.ntq - r.t0;
        r.s0 = 0;
        r.s1 = r.span * sp.group;
    }
    return r;
}

// Float offset of partial `slot` (0: the sink tile's band unit, 1 + c: chunk c) of
// key/value head bh: dK rows, then dV rows.
__host__ __device__ inline size_t sink_partial_offset(const SinkSplit& sp, int bh, int slot, int d) {
    if (sp.chunks == 0) return 0;
    return ((size_t)bh * (sp.chunks + 1) + slot) * 2 * sp.rows * d;
}

inline size_t sink_delta_bytes(int B, int Hq, int N) { return ((size_t)B * Hq * N * 4 + 255) / 256 * 256; }

// Adds the partials of the sink tokens' dk, dv in the order of their slots.
template <typename E>
cudaError_t launch_sink_join(const SinkArgs& a, const SinkSplit& sp, const float* partial, cudaStream_t stream);

}  // namespace based
