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
            s = 0.f;
            constexpr int P = 16 / (int)sizeof(E);           // channels of a 16-byte piece
#pragma unroll 1
            for (int c = 0; c < D; c += 4 * P) {             // the loads of four pieces in flight
                uint4 a[4], b[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    a[x] = *reinterpret_cast<const uint4*>(q + c + x * P);
                    b[x] = *reinterpret_cast<const uint4*>(kr + c + x * P);
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) s = dot16(a[x], b[x], s, q);
            }
            s *= scale;
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
