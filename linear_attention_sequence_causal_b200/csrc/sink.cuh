// Shared by the kernels of the sliding-window attention with sink tokens.
#pragma once

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace based {

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

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xFFFF0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// How the dK, dV work of one key/value head is cut into units, for tiles of T
// rows: nt band units (key tile kt against the query tiles that see it through the
// window, over the group's heads) and `chunks` units of the sink tile, each a
// stretch of `chunk_len` steps of the list (head of the group, query tile past the
// window). A chunk is as long as a full band unit, so the units stay even.
struct SinkSplit {
    int nt, chunks, chunk_len, span, t_first, band, group;
    int rows;                                // rows of a partial: the sink tokens
    __host__ __device__ int units() const { return nt + chunks; }
};

inline SinkSplit sink_split(int Hq, int Hkv, int N, int w, int n_sink, int T) {
    SinkSplit s{};
    s.nt = (N + T - 1) / T;
    s.group = Hq / Hkv;
    s.rows = n_sink;
    s.band = (int)std::min<long long>(s.nt, ((long long)w + T - 2) / T + 1);
    if (n_sink > 0 && w < N) {               // a query i >= w has sinks outside its window
        s.t_first = w / T;
        s.span = s.nt - s.t_first;
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
__host__ __device__ inline SinkUnit sink_unit(const SinkSplit& sp, int u, int B, int Hkv) {
    SinkUnit r;
    const int bh = u % (B * Hkv), i = u / (B * Hkv);
    r.b = bh / Hkv;
    r.hk = bh % Hkv;
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
        r.t0 = r.kt;
        r.span = r.kt + sp.band <= sp.nt ? sp.band : sp.nt - r.kt;
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
