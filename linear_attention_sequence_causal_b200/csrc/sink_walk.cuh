// What the blocks of the bf16 backward work through: units, their steps, and which pairs a
// step sees. Runs on the host too, where a test walks every unit.
#pragma once

#include "sink.cuh"

namespace based {

constexpr int kOwnRows = 128;                // rows of a unit's own tile

__host__ __device__ inline int clamped_len(const int64_t* lengths, int b, int N) {
    if (lengths == nullptr) return N;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : n > N ? N : (int)n;
}

// Queries [from, end) that see key j in a DKV step: [j, j + w) in a band unit, [j + w, ..) of
// a sink in a chunk; none past the sequence's end.
struct QueryRange {
    int from, end;
    __host__ __device__ inline QueryRange(bool chunk, int j, int len, int w, int n_sink)
        : from(chunk ? (j < n_sink ? j + w : 0x7fffffff) : j), end(chunk ? len : min(len, j + w)) {}
};

// What a step is, in shared memory beside its ring stage (written before the stage's
// copies are announced, read once A has landed).
struct Head {
    enum { kLast = 1, kSink = 2, kEnd = 4, kFirst = 8, kScan = 16, kScanEnd = 32 };
    // kLast: of the unit; kSink: the sink block; kEnd: of the block's work.
    // kFirst: the unit's first product; kScan: a step of the sweep for delta, kScanEnd: its last.
    int own, ring, len, flags;               // first rows of the own tile and of the step, tokens
    int b, head, tag, pad;                   // of the own tile; DKV: chunk or -1
};
static_assert(sizeof(Head) == 32, "header");

// A walk over the units of a block and their steps, which the loading thread takes; the
// other roles read what they need of it from the header of each ring stage (Head).
// Steps: DQ the sink block (t = -1), then key tiles lo .. hi; DKV the pairs (head, query
// tile) of the unit's stretch, without tiles of padding. A unit with nothing to compute
// (padding) keeps one step, in which no row sees anything.
template <int W>
struct DqWalk {
    int u, b, h, hk, own, lo, hi, len;       // own: first query
    int t, t0;                               // the current step's key tile, -1: the sink block; the first one's
    bool scan;                               // in the sweep for delta (see above)

    template <typename P>
    __host__ __device__ inline void start(const P& p, int unit) {
        u = unit;
        if (u >= p.units) return;
        const int x = p.by_bhq.div(u), bh = u - x * (int)p.by_bhq.d;
        own = (p.nt - 1 - x) * kOwnRows;     // long sweeps first
        b = p.by_hq.div(bh);
        h = bh - b * p.Hq;
        hk = p.by_group.div(h);
        len = clamped_len(p.lengths, b, p.N);
        lo = max(0, own - p.w + 1) / W;
        hi = own < len ? (min(own + kOwnRows, len) - 1) / W : lo;
        t = t0 = own < len && p.n_sink > 0 && lo > 0 ? -1 : lo;
        scan = own < len && min(own + 1, p.w + p.n_sink) < 64;
    }
    __host__ __device__ inline bool last() const { return t == hi && !scan; }
    __host__ __device__ inline void next() {
        if (t == hi) {
            scan = false;
            t = t0;
        } else {
            t = t < 0 ? lo : t + 1;
        }
    }
    __host__ __device__ inline int sweep() const {
        return scan ? Head::kScan | (t == hi ? Head::kScanEnd : 0) : t == t0 ? Head::kFirst : 0;
    }
    __host__ __device__ inline bool sink() const { return t < 0; }
    __host__ __device__ inline int own_head() const { return h; }
    __host__ __device__ inline int ring_head() const { return hk; }
    __host__ __device__ inline int ring_row() const { return t < 0 ? 0 : t * W; }
    __host__ __device__ inline int tag() const { return 0; }
};

template <int W>
struct KvWalk {
    int u, b, hk, own, chunk, len;           // own: first key
    int h, t;                                // the current step: query head and tile
    int t0, tv, left, span;                  // tiles t0 .. tv - 1 are real; list entries left (this one too)
    bool first;                              // the unit's first step

    template <typename P>
    __host__ __device__ inline void start(const P& p, int unit) {
        u = unit;
        first = true;
        if (u >= p.units) return;
        const SinkUnit x = sink_unit(p.sp, u, p.by_bhkv, p.by_hkv);
        b = x.b, hk = x.hk, own = x.kt * kOwnRows, chunk = x.chunk;
        len = clamped_len(p.lengths, b, p.N);
        t0 = x.t0;
        span = x.span;
        tv = min(x.t0 + x.span, (len + W - 1) / W);
        const int skip_heads = chunk > 0 ? x.s0 / x.span : 0;
        h = hk * p.sp.group + skip_heads;
        t = x.t0 + x.s0 - skip_heads * x.span;
        left = x.s1 - x.s0;
        if (t >= tv) skip();
        if (tv <= t0 || own >= len || left <= 0) {           // nothing: one step, all hidden
            // by a length of 0, whatever the tile holds: a stretch may be all padding in a
            // sequence that has real tiles.
            len = 0;
            h = hk * p.sp.group;
            t = t0;
            tv = t0 + 1;
            left = 1;
        }
    }
    __host__ __device__ inline void skip() {                 // to the next head's first tile
        left -= t0 + span - t;
        t = t0;
        ++h;
    }
    // Entries after this one: in this head, or (with at least one real tile) in a later one.
    __host__ __device__ inline bool last() const { return t + 1 < tv ? left <= 1 : left - (t0 + span - t) <= 0; }
    __host__ __device__ inline int sweep() const { return first ? Head::kFirst : 0; }
    __host__ __device__ inline void next() {
        first = false;
        if (t + 1 < tv) {
            ++t;
            --left;
        } else {
            skip();
        }
    }
    __host__ __device__ inline bool sink() const { return false; }
    __host__ __device__ inline int own_head() const { return hk; }
    __host__ __device__ inline int ring_head() const { return h; }
    __host__ __device__ inline int ring_row() const { return t * W; }
    __host__ __device__ inline int tag() const { return chunk; }
};

}  // namespace based
