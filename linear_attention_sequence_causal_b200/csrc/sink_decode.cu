// One generated token per sequence over the sink + ring cache.
//
// The cache rows in use are read once, so memory bounds the step. A block of 4 or 8
// warps takes up to 16 of the query heads that share a key/value head; each warp
// streams its own stages of 16 slots (K and V rows) by TMA into a private ring, with
// no block-wide wait until the end, and keeps the running maximum, sum and
// accumulator of a softmax. bf16: both products are 16 x 8 x 16 matrix instructions
// (rows = heads), so their cost does not grow with the group; fp32: multiply-adds,
// heads in registers. A long window is split over a cluster of up to 16 blocks; the
// blocks' (maximum, sum, accumulator) are joined through distributed shared memory in
// a fixed order. (Copies by cp.async, 16 per lane and stage, kept an SM at 32 bytes a
// cycle whatever the ring's depth: one sequence at w = 32768, 4 heads of 128 took 34 us.)
//
// 64 sequences of 16 heads over 4 x 1028 slots of 128: 113 MB in 23.6 us (4.8 TB/s of 6.55);
// one sequence, 32784 slots: 67 MB in 22.2 us (3.0 TB/s: 64 blocks in clusters of 16 land
// on half of the chip's SM groups); one sequence, 68 slots: 3.5 us, a launch's latency. fp32:
// 270 MB of the first in 326 us (0.83 TB/s: the rings leave an SM four warps, whose chains of
// multiply-adds wait on themselves, and a third of them is for heads that are not there). The
// stages of all sequences as one list, cut evenly over the SMs and joined by a second
// launch, took 43 us on the first of these.
#include <algorithm>

#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"
#include "tcgen05_heads.cuh"
#include "tma_host.h"

namespace based {
namespace {

namespace cg = cooperative_groups;
using tc::smem_u32;

constexpr int kStageSlots = 16;
constexpr int kStages = 3;                   // ring stages per warp
constexpr int kHeads = 16;                   // query heads per block (rows of the matrix instruction)
constexpr int kMaxSplit = 16;

struct DecodeArgs {
    void* kc;
    void* vc;
    const int64_t* positions;
    const void* q;
    const void* k;
    const void* v;
    void* y;
    unsigned* status;
    int Hq, Hkv, w, n_sink, head_blocks, split;
    float scale;
};

template <typename E, int D, int WARPS>
struct DecodeLayout {
    static constexpr int ROW = D * (int)sizeof(E);               // bytes
    static constexpr int PIECES = ROW / 16;
    static constexpr int STAGE = 2 * kStageSlots * ROW;          // K, then V
    static constexpr int BLOCK = kStageSlots * 128;              // 128 bytes of 16 rows, 128-byte swizzle
    static constexpr int RING = WARPS * kStages * STAGE;
    // After the sweep the ring holds every warp's accumulator, then the block's.
    static constexpr int ACC = kHeads * D * 4;
    static_assert(RING >= WARPS * ACC, "accumulators fit the ring");
    static constexpr int OFF_ML = RING;                          // per warp: m[16], l[16]; then the block's
    static constexpr int OFF_BAR = OFF_ML + (WARPS + 1) * 2 * kHeads * 4;
    static constexpr int SMEM = OFF_BAR + WARPS * kStages * 8 + 8 + 1024;   // + the abort flag, alignment slack
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void ldmatrix4(uint32_t* r, uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t* r, uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Offset of 16-byte piece p of slot row r in a stage's K or V: blocks of 128 bytes by 16
// rows whose pieces the copy permutes by the row, so that 8 rows read at one column hit
// 8 different bank groups.
__device__ __forceinline__ uint32_t piece_at(int r, int p) {
    return (uint32_t)((p >> 3) * (kStageSlots * 128) + r * 128 + (((p & 7) ^ (r & 7)) << 4));
}

// What a block works on.
struct Where {
    int b, hk, h0, nh;           // sequence, key/value head, first query head, query heads
    int rank, split;
    int n, slot;                 // slots in use (with the new token), the new token's slot
    long long kv_row;            // row of (b, hk) in k, v
    bool writes;                 // stores the new token into the cache
};

__device__ __forceinline__ Where where(const DecodeArgs& a) {
    Where w;
    w.split = a.split;
    w.rank = blockIdx.x % a.split;
    int u = blockIdx.x / a.split;
    const int hb = u % a.head_blocks;
    u /= a.head_blocks;
    w.hk = u % a.Hkv;
    w.b = u / a.Hkv;
    const int group = a.Hq / a.Hkv;
    w.h0 = w.hk * group + hb * kHeads;
    w.nh = min(kHeads, group - hb * kHeads);
    w.kv_row = (long long)w.b * a.Hkv + w.hk;
    w.writes = hb == 0;
    const int64_t t = a.positions[w.b];
    if (t < 0) {
        w.n = 0;
        w.slot = -1;
    } else if (t < a.n_sink) {
        w.n = (int)t + 1;
        w.slot = (int)t;
    } else {
        const int64_t past = t - a.n_sink;
        w.n = a.n_sink + (int)(past + 1 < a.w ? past + 1 : a.w);
        w.slot = a.n_sink + (int)(past % a.w);
    }
    return w;
}

// Issues the copies of stage s (slots 16 s ..) of this block's cache rows: one lane.
template <typename E, int D, int WARPS>
__device__ __forceinline__ void issue_stage(uint32_t dst, uint64_t* bar, const CUtensorMap* mk, const CUtensorMap* mv,
                                            const Where& w, int s) {
    using L = DecodeLayout<E, D, WARPS>;
    tc::mbar_expect_tx(bar, L::STAGE);
#pragma unroll
    for (int h = 0; h < L::ROW / 128; ++h) {
        tc::tma_load_4d(dst + h * L::BLOCK, mk, bar, 64 * h, s * kStageSlots, w.hk, w.b);
        tc::tma_load_4d(dst + L::STAGE / 2 + h * L::BLOCK, mv, bar, 64 * h, s * kStageSlots, w.hk, w.b);
    }
}

// Puts the new token's k, v into its row of the landed stage, and into the cache; rows of
// V from `n` on, which no weight may meet whatever they hold, become zeros.
template <typename E, int D, int WARPS>
__device__ __forceinline__ void patch_stage(const DecodeArgs& a, const Where& w, uint32_t stage, int s, int lane) {
    using L = DecodeLayout<E, D, WARPS>;
    if (w.slot / kStageSlots == s) {
        const uint4* k = reinterpret_cast<const uint4*>(static_cast<const char*>(a.k) + w.kv_row * L::ROW);
        const uint4* v = reinterpret_cast<const uint4*>(static_cast<const char*>(a.v) + w.kv_row * L::ROW);
        const long long row = (w.kv_row * ((long long)a.n_sink + a.w) + w.slot) * L::PIECES;
        for (int p = lane; p < L::PIECES; p += 32) {
            const uint4 kp = k[p], vp = v[p];
            tc::st_shared_v4(stage + piece_at(w.slot % kStageSlots, p), kp);
            tc::st_shared_v4(stage + L::STAGE / 2 + piece_at(w.slot % kStageSlots, p), vp);
            if (w.writes) {
                static_cast<uint4*>(a.kc)[row + p] = kp;
                static_cast<uint4*>(a.vc)[row + p] = vp;
            }
        }
    }
    for (int i = lane; i < kStageSlots * L::PIECES; i += 32)
        if (s * kStageSlots + i / L::PIECES >= w.n)
            tc::st_shared_v4(stage + L::STAGE / 2 + piece_at(i / L::PIECES, i % L::PIECES), make_uint4(0, 0, 0, 0));
    tc::fence_proxy_async_smem();                            // before a later copy lands in the same place
    __syncwarp();
}

// The running softmax of one warp, bf16: rows lane / 4 and lane / 4 + 8 of the heads.
// The weights are the second product's A operand, in two bf16 parts: cut off, and what that
// leaves, rounded, so that 2^-15 of a weight is lost (one rounded part: 2^-8, an error of
// 0.0022 of y's size, of which y's own rounding makes 0.0017). The second part is never below
// kLeast: beside a first part that makes an infinite value infinite, 0 or a negative number
// would make it NaN. HALF (at most 8 heads): the second parts take the rows that heads leave
// free and cost nothing; else a second product adds them (64 x 16 heads over 4 x 1028 slots
// of 128, us: 24.4 for one part, 26.1 for two products, 23.6 for two parts in one).
template <int D, bool HALF>
struct WarpBf16 {
    static constexpr int V_OFF = kStageSlots * D * 2;            // V behind K in a stage
    static constexpr int ROWS = HALF ? 1 : 2;                    // heads per lane
    static constexpr float kLeast = 2.4e-38f;                    // a normal number in bf16 too
    uint32_t q[D / 16][4];
    float o[D / 8][4], m[2], l[2];

    __device__ __forceinline__ void init(const DecodeArgs& a, const Where& w, int lane) {
        const __nv_bfloat16* q0 = static_cast<const __nv_bfloat16*>(a.q) + ((long long)w.b * a.Hq + w.h0) * D;
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = lane / 4 + 8 * (e & 1), c = 16 * j + 2 * (lane % 4) + 8 * (e >> 1);
                q[j][e] = r < w.nh ? *reinterpret_cast<const uint32_t*>(q0 + r * D + c) : 0u;
            }
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }

    __device__ __forceinline__ void step(uint32_t st, int slot0, int n, float scale_log2, int lane) {
        float s[2][4] = {};
        const int mr = lane & 7, mi = lane >> 3;             // ldmatrix: row and matrix of this lane's address
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            uint32_t b[4];
            ldmatrix4(b, st + piece_at(mr + 8 * (mi >> 1), 2 * j + (mi & 1)));
            mma16816(s[0], q[j], b[0], b[1]);
            mma16816(s[1], q[j], b[2], b[3]);
        }
        float p[2][4];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            float x[4];
            float mx = -INFINITY;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = slot0 + 2 * (lane % 4) + (e & 1) + 8 * (e >> 1);
                x[e] = key < n ? s[e >> 1][2 * r + (e & 1)] * scale_log2 : -INFINITY;
                mx = fmaxf(mx, x[e]);
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float mn = fmaxf(m[r], mx);
            const float mu = mn == -INFINITY ? 0.f : mn;
            if (__any_sync(0xffffffffu, mn > m[r])) {
                const float al = exp2f(m[r] - mu);
                l[r] *= al;
#pragma unroll
                for (int j = 0; j < D / 8; ++j)
#pragma unroll
                    for (int e = 2 * r; e < 2 * r + 4 / ROWS; ++e) o[j][e] *= al;
            }
            m[r] = mn;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                p[r][e] = exp2f(x[e] - mu);
                l[r] += p[r][e];
            }
        }
        // A operand: rows lane / 4 (+ 8), keys 2 (lane % 4) (+ 8).
        uint32_t pa[4], rest[4];
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                pa[e + r] = __byte_perm(__float_as_uint(p[r][e]), __float_as_uint(p[r][e + 1]), 0x7632);   // the upper halves
                rest[e + r] = tc::pack_bf16x2(fmaxf(p[r][e] - __uint_as_float(pa[e + r] << 16), kLeast),
                                              fmaxf(p[r][e + 1] - __uint_as_float(pa[e + r] & 0xFFFF0000u), kLeast));
            }
        if (HALF) pa[1] = rest[0], pa[3] = rest[2];
        const uint32_t sv = st + V_OFF;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            uint32_t b[4];
            ldmatrix4_t(b, sv + piece_at(mr + 8 * (mi & 1), 2 * j + (mi >> 1)));
            mma16816(o[2 * j], pa, b[0], b[1]);
            mma16816(o[2 * j + 1], pa, b[2], b[3]);
            if (!HALF) {
                mma16816(o[2 * j], rest, b[0], b[1]);
                mma16816(o[2 * j + 1], rest, b[2], b[3]);
            }
        }
    }

    __device__ __forceinline__ void store(float* acc, float* ml, int lane) {
        if (HALF) {
#pragma unroll
            for (int j = 0; j < D / 8; ++j) o[j][0] += o[j][2], o[j][1] += o[j][3];
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            const int h = lane / 4 + 8 * r;
            if (lane % 4 == 0) {
                ml[h] = m[r];
                ml[kHeads + h] = l[r];
            }
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
                *reinterpret_cast<float2*>(acc + h * D + 8 * j + 2 * (lane % 4)) =
                    make_float2(o[j][2 * r], o[j][2 * r + 1]);
        }
    }
};

// fp32: lane holds key lane % 16 (half lane / 16 of the channels) for the scores and
// channels lane * D / 32 .. for the accumulators. Queries are read from global
// memory (a few KB, in L1).
template <int D>
struct WarpF32 {
    static constexpr int V_OFF = kStageSlots * D * 4;
    static constexpr int CH = D / 32;
    const float* q;
    int nh;
    float o[kHeads][CH], m[kHeads], l[kHeads];

    __device__ __forceinline__ void init(const DecodeArgs& a, const Where& w, int lane) {
        q = static_cast<const float*>(a.q) + ((long long)w.b * a.Hq + w.h0) * D;
        nh = w.nh;
#pragma unroll
        for (int g = 0; g < kHeads; ++g) {
            m[g] = -INFINITY, l[g] = 0.f;
#pragma unroll
            for (int c = 0; c < CH; ++c) o[g][c] = 0.f;
        }
    }

    __device__ __forceinline__ void step(uint32_t st, int slot0, int n, float scale_log2, int lane) {
        const int key = lane & 15, half = lane >> 4;
        const bool live = slot0 + key < n;
        float s[kHeads];
#pragma unroll
        for (int g = 0; g < kHeads; ++g) s[g] = 0.f;
        for (int p = half * (D / 8); p < (half + 1) * (D / 8); ++p) {      // 16-byte pieces
            const uint4 kr = tc::ld_shared_v4(st + piece_at(key, p));
#pragma unroll
            for (int g = 0; g < kHeads; ++g)
                if (g < nh) {
                    const float4 qr = __ldg(reinterpret_cast<const float4*>(q + g * D + 4 * p));
                    s[g] = fmaf(__uint_as_float(kr.x), qr.x, s[g]);
                    s[g] = fmaf(__uint_as_float(kr.y), qr.y, s[g]);
                    s[g] = fmaf(__uint_as_float(kr.z), qr.z, s[g]);
                    s[g] = fmaf(__uint_as_float(kr.w), qr.w, s[g]);
                }
        }
#pragma unroll
        for (int g = 0; g < kHeads; ++g)
            if (g < nh) {
                float x = s[g] + __shfl_xor_sync(0xffffffffu, s[g], 16);
                x = live ? x * scale_log2 : -INFINITY;
                float mx = x;
#pragma unroll
                for (int b = 8; b > 0; b >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, b));
                const float mn = fmaxf(m[g], mx);
                const float mu = mn == -INFINITY ? 0.f : mn;
                const float al = exp2f(m[g] - mu);
                s[g] = exp2f(x - mu);
                l[g] = l[g] * al + (half == 0 ? s[g] : 0.f);         // per lane; summed at the end
                m[g] = mn;
#pragma unroll
                for (int c = 0; c < CH; ++c) o[g][c] *= al;
            }
        const uint32_t sv = st + V_OFF;
#pragma unroll 4
        for (int r = 0; r < kStageSlots; ++r) {
            float v[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int byte = (lane * CH + c) * 4;
                v[c] = tc::ld_shared_f32(sv + piece_at(r, byte >> 4) + (byte & 15));
            }
#pragma unroll
            for (int g = 0; g < kHeads; ++g)
                if (g < nh) {
                    const float p = __shfl_sync(0xffffffffu, s[g], r);
#pragma unroll
                    for (int c = 0; c < CH; ++c) o[g][c] = fmaf(p, v[c], o[g][c]);
                }
        }
    }

    __device__ __forceinline__ void store(float* acc, float* ml, int lane) {
#pragma unroll
        for (int g = 0; g < kHeads; ++g) {
            float t = l[g];
#pragma unroll
            for (int b = 16; b > 0; b >>= 1) t += __shfl_xor_sync(0xffffffffu, t, b);
            if (lane == 0) {
                ml[g] = m[g];
                ml[kHeads + g] = t;
            }
#pragma unroll
            for (int c = 0; c < CH; ++c) acc[g * D + lane * CH + c] = o[g][c];
        }
    }
};

template <typename E, int D, bool HALF> struct WarpOf { using type = WarpBf16<D, HALF>; };
template <int D, bool HALF> struct WarpOf<float, D, HALF> { using type = WarpF32<D>; };

template <typename E, int D, int WARPS, bool HALF>
__global__ void __launch_bounds__(WARPS * 32)
sink_decode_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                   const __grid_constant__ DecodeArgs a) {
    using L = DecodeLayout<E, D, WARPS>;
    extern __shared__ unsigned char smem_raw[];
    // The same offset in every block of a cluster: the join addresses the others' memory by it.
    unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_BAR + WARPS * kStages * 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < WARPS * kStages; ++i) tc::mbar_init(&bars[i], 1);
        *abort_flag = 0;
        tc::mbar_fence_init();
        tc::prefetch_tensormap(&mk);
        tc::prefetch_tensormap(&mv);
    }
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();
    const Where w = where(a);
    const float scale_log2 = a.scale * 1.44269504088896340736f;
    const uint32_t ring = smem_u32(smem) + warp * kStages * L::STAGE;
    uint64_t* bar = bars + warp * kStages;
    const int stages = (w.n + kStageSlots - 1) / kStageSlots;
    const int first = w.rank * WARPS + warp, stride = w.split * WARPS;
    const int mine = first < stages ? (stages - first + stride - 1) / stride : 0;    // stages of this warp
    typename WarpOf<E, D, HALF>::type acc;
    if (lane == 0)
        for (int i = 0; i < kStages && i < mine; ++i)
            issue_stage<E, D, WARPS>(ring + i * L::STAGE, bar + i, &mk, &mv, w, first + i * stride);
    acc.init(a, w, lane);
    int done = 0;
    for (; done < mine; ++done) {
        const int buf = done % kStages, s = first + done * stride;
        if (!__all_sync(0xffffffffu, tc::mbar_wait(bar + buf, (done / kStages) & 1, abort_flag, a.status))) break;
        const uint32_t st = ring + buf * L::STAGE;
        if (w.slot / kStageSlots == s || (s + 1) * kStageSlots > w.n) patch_stage<E, D, WARPS>(a, w, st, s, lane);
        acc.step(st, s * kStageSlots, w.n, scale_log2, lane);
        __syncwarp();                                        // the stage may be refilled
        if (lane == 0 && done + kStages < mine)
            issue_stage<E, D, WARPS>(st, bar + buf, &mk, &mv, w, s + kStages * stride);
    }
    // After a copy that never landed: wait (bounded) for it and the ones behind it.
    for (int i = done; i < mine && i < done + kStages; ++i) {
        const uint64_t t0 = global_ns();
        while (!tc::mbar_try_wait(bar + i % kStages, (i / kStages) & 1) && global_ns() - t0 < kWaitLimitNs) {}
    }
    __syncthreads();                                         // the ring becomes the accumulators' store
    float* accs = reinterpret_cast<float*>(smem);
    float* ml = reinterpret_cast<float*>(smem + L::OFF_ML);
    acc.store(accs + warp * kHeads * D, ml + warp * 2 * kHeads, lane);
    __syncthreads();
    // Join the warps: the block's accumulator over warp 0's, its (m, l) behind the warps'.
    float* bml = ml + WARPS * 2 * kHeads;
    for (int i = threadIdx.x; i < w.nh * D; i += WARPS * 32) {
        const int h = i / D;
        float mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < WARPS; ++k) mx = fmaxf(mx, ml[k * 2 * kHeads + h]);
        const float mu = mx == -INFINITY ? 0.f : mx;
        float x = 0.f, sum = 0.f;
#pragma unroll
        for (int k = 0; k < WARPS; ++k) {
            const float f = exp2f(ml[k * 2 * kHeads + h] - mu);
            x = fmaf(f, accs[k * kHeads * D + i], x);
            sum = fmaf(f, ml[k * 2 * kHeads + kHeads + h], sum);
        }
        accs[i] = x;
        if (i % D == 0) {
            bml[h] = mx;
            bml[kHeads + h] = sum;
        }
    }
    E* y = static_cast<E*>(a.y) + ((long long)w.b * a.Hq + w.h0) * D;
    if (w.split == 1) {
        __syncthreads();
        for (int i = threadIdx.x; i < w.nh * D; i += WARPS * 32)
            y[i] = from_f32<E>(w.n > 0 ? accs[i] / bml[kHeads + i / D] : 0.f);
        return;
    }
    // Join the cluster's blocks: block `rank` writes its share of the outputs.
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    for (int i = w.rank * WARPS * 32 + threadIdx.x; i < w.nh * D; i += w.split * WARPS * 32) {
        const int h = i / D;
        float mk[kMaxSplit];
        float mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < kMaxSplit; ++k) {
            mk[k] = k < w.split ? cluster.map_shared_rank(bml, k)[h] : -INFINITY;
            mx = fmaxf(mx, mk[k]);
        }
        const float mu = mx == -INFINITY ? 0.f : mx;
        float x = 0.f, sum = 0.f;
#pragma unroll
        for (int k = 0; k < kMaxSplit; ++k)
            if (k < w.split) {
                const float f = exp2f(mk[k] - mu);
                x = fmaf(f, cluster.map_shared_rank(accs, k)[i], x);
                sum = fmaf(f, cluster.map_shared_rank(bml, k)[kHeads + h], sum);
            }
        y[i] = from_f32<E>(w.n > 0 ? x / sum : 0.f);
    }
    cluster.sync();                                          // no block leaves while another reads its memory
}

// Blocks per (sequence, key/value head, 16 heads): doubled while the blocks do not fill
// the SMs (two blocks of 4 warps each) and each warp keeps at least 2 stages of a full window.
int plan_split(long long base, int slots, int num_sms) {
    int split = 1;
    while (split < kMaxSplit && base * split * 2 <= 2LL * num_sms && slots >= split * 2 * 4 * kStageSlots * 2) split *= 2;
    return split;
}

template <typename E, int D, int WARPS, bool HALF>
cudaError_t run(const DecodeArgs& a, int B, long long blocks, cudaStream_t stream) {
    using L = DecodeLayout<E, D, WARPS>;
    auto kern = sink_decode_kernel<E, D, WARPS, HALF>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e == cudaSuccess && a.split > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    // The rows' bytes as 16-bit elements: a copy does not look at them.
    const uint64_t x = L::ROW / 2, slots = (uint64_t)a.n_sink + a.w;
    CUtensorMap mk, mv;
    if (!make_tmap_bf16_heads(&mk, a.kc, x, slots, a.Hkv, B, x, x * slots, x * slots * a.Hkv, kStageSlots) ||
        !make_tmap_bf16_heads(&mv, a.vc, x, slots, a.Hkv, B, x, x * slots, x * slots * a.Hkv, kStageSlots))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(WARPS * 32);
    cfg.dynamicSmemBytes = L::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, mk, mv, a);
}

template <typename E, int D>
cudaError_t pick(DecodeArgs a, int B, int num_sms, cudaStream_t stream) {
    a.head_blocks = (a.Hq / a.Hkv + kHeads - 1) / kHeads;
    const long long base = (long long)B * a.Hkv * a.head_blocks;
    a.split = plan_split(base, a.n_sink + a.w, num_sms);
    if (base * a.split > 0x7fffffffLL) return cudaErrorInvalidValue;
    const long long blocks = base * a.split;
    // At most one block per SM: 8 warps keep twice the bytes in flight there (one sequence,
    // 32784 slots, 4 x 128: 23 us against 33 with 4 warps; beyond, two blocks share an SM).
    if constexpr (sizeof(E) == 2) {
        const bool half = a.Hq / a.Hkv <= kHeads / 2;
        if (blocks <= num_sms) return half ? run<E, D, 8, true>(a, B, blocks, stream) : run<E, D, 8, false>(a, B, blocks, stream);
        if (half) return run<E, D, 4, true>(a, B, blocks, stream);
    }
    return run<E, D, 4, false>(a, B, blocks, stream);
}

}  // namespace

cudaError_t launch_sink_decode(void* k_cache, void* v_cache, const int64_t* positions, const void* q, const void* k,
                               const void* v, void* y, int B, int Hq, int Hkv, int d, int w, int n_sink, float scale,
                               bool bf16, int num_sms, unsigned* status, cudaStream_t stream) {
    const DecodeArgs a{k_cache, v_cache, positions, q, k, v, y, status, Hq, Hkv, w, n_sink, 1, 1, scale};
    if (bf16)
        return d == 64 ? pick<__nv_bfloat16, 64>(a, B, num_sms, stream) : pick<__nv_bfloat16, 128>(a, B, num_sms, stream);
    return d == 64 ? pick<float, 64>(a, B, num_sms, stream) : pick<float, 128>(a, B, num_sms, stream);
}

}  // namespace based
