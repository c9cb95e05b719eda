// One generated token per sequence over the sink + ring cache.
//
// The cache rows in use are read once, so memory bounds the step. A block of 4
// warps takes up to 16 of the query heads that share a key/value head; each warp
// streams its own stages of 16 slots (K and V rows) through a private ring of
// cp.async stages, with no block-wide wait until the end, and keeps the running
// maximum, sum and accumulator of a softmax. bf16: both products are 16 x 8 x 16
// matrix instructions (rows = heads), so their cost does not grow with the group;
// fp32: multiply-adds, heads in registers. A long window is split over a cluster of
// up to 16 blocks; the blocks' (maximum, sum, accumulator) are joined through
// distributed shared memory in a fixed order.
#include <algorithm>

#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace based {
namespace {

namespace cg = cooperative_groups;
using tc::smem_u32;

constexpr int kWarps = 4;
constexpr int kStageSlots = 16;
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
    int Hq, Hkv, w, n_sink, head_blocks, split;
    float scale;
};

template <typename E, int D>
struct DecodeLayout {
    static constexpr int ROW = D * (int)sizeof(E);               // bytes
    static constexpr int PIECES = ROW / 16;
    static constexpr int STAGE = 2 * kStageSlots * ROW;          // K, then V
    static constexpr int STAGES = sizeof(E) == 2 ? (D == 128 ? 3 : 4) : 2;
    static constexpr int RING = kWarps * STAGES * STAGE;
    // After the sweep the ring holds every warp's accumulator, then the block's.
    static constexpr int ACC = kHeads * D * 4;
    static constexpr int OFF_ML = RING > kWarps * ACC ? RING : kWarps * ACC;   // per warp: m[16], l[16]
    static constexpr int SMEM = OFF_ML + (kWarps + 1) * 2 * kHeads * 4;        // the last: the block's
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
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

// Shared-memory offset of 16-byte piece p of slot row r: pieces XOR-permuted within
// 128 bytes, so that 8 rows read at one column hit 8 different bank groups.
template <int ROW>
__device__ __forceinline__ uint32_t piece_at(int r, int p) {
    return (uint32_t)(r * ROW + ((p ^ (r & 7)) << 4));
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

// Issues the copies of stage s (slots 16 s ..; slots not in use are zero-filled).
template <typename E, int D>
__device__ __forceinline__ void issue_stage(uint32_t dst, const char* kc, const char* vc, int s, int n, int lane) {
    using L = DecodeLayout<E, D>;
#pragma unroll
    for (int i = lane; i < kStageSlots * L::PIECES; i += 32) {
        const int r = i / L::PIECES, p = i % L::PIECES;
        const int slot = s * kStageSlots + r;
        const bool live = slot < n;
        const long long off = (long long)(live ? slot : 0) * L::ROW + 16 * p;
        cp_async16(dst + piece_at<L::ROW>(r, p), kc + off, live);
        cp_async16(dst + kStageSlots * L::ROW + piece_at<L::ROW>(r, p), vc + off, live);
    }
}

// Puts the new token's k, v into its row of the landed stage, and into the cache.
template <typename E, int D>
__device__ __forceinline__ void put_token(const DecodeArgs& a, const Where& w, uint32_t stage, int r, char* kc,
                                          char* vc, int lane) {
    using L = DecodeLayout<E, D>;
    const uint4* k = reinterpret_cast<const uint4*>(static_cast<const char*>(a.k) + w.kv_row * L::ROW);
    const uint4* v = reinterpret_cast<const uint4*>(static_cast<const char*>(a.v) + w.kv_row * L::ROW);
    for (int p = lane; p < L::PIECES; p += 32) {
        const uint4 kp = k[p], vp = v[p];
        tc::st_shared_v4(stage + piece_at<L::ROW>(r, p), kp);
        tc::st_shared_v4(stage + kStageSlots * L::ROW + piece_at<L::ROW>(r, p), vp);
        if (w.writes) {
            reinterpret_cast<uint4*>(kc + (long long)w.slot * L::ROW)[p] = kp;
            reinterpret_cast<uint4*>(vc + (long long)w.slot * L::ROW)[p] = vp;
        }
    }
    __syncwarp();
}

// The running softmax of one warp, bf16: rows lane / 4 and lane / 4 + 8 of the heads.
template <int D>
struct WarpBf16 {
    using L = DecodeLayout<__nv_bfloat16, D>;
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
            ldmatrix4(b, st + piece_at<L::ROW>(mr + 8 * (mi >> 1), 2 * j + (mi & 1)));
            mma16816(s[0], q[j], b[0], b[1]);
            mma16816(s[1], q[j], b[2], b[3]);
        }
        float p[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
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
                for (int j = 0; j < D / 8; ++j) {
                    o[j][2 * r] *= al;
                    o[j][2 * r + 1] *= al;
                }
            }
            m[r] = mn;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                p[r][e] = exp2f(x[e] - mu);
                l[r] += p[r][e];
            }
        }
        // The weights as the A operand (bf16): rows lane / 4 (+ 8), keys 2 (lane % 4) (+ 8).
        const uint32_t pa[4] = {tc::pack_bf16x2(p[0][0], p[0][1]), tc::pack_bf16x2(p[1][0], p[1][1]),
                                tc::pack_bf16x2(p[0][2], p[0][3]), tc::pack_bf16x2(p[1][2], p[1][3])};
        const uint32_t sv = st + kStageSlots * L::ROW;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            uint32_t b[4];
            ldmatrix4_t(b, sv + piece_at<L::ROW>(mr + 8 * (mi & 1), 2 * j + (mi >> 1)));
            mma16816(o[2 * j], pa, b[0], b[1]);
            mma16816(o[2 * j + 1], pa, b[2], b[3]);
        }
    }

    __device__ __forceinline__ void store(float* acc, float* ml, int lane) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
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
    using L = DecodeLayout<float, D>;
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
            const uint4 kr = tc::ld_shared_v4(st + piece_at<L::ROW>(key, p));
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
        const uint32_t sv = st + kStageSlots * L::ROW;
#pragma unroll 4
        for (int r = 0; r < kStageSlots; ++r) {
            float v[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int byte = (lane * CH + c) * 4;
                v[c] = tc::ld_shared_f32(sv + piece_at<L::ROW>(r, byte >> 4) + (byte & 15));
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

template <typename E, int D> struct WarpOf;
template <int D> struct WarpOf<__nv_bfloat16, D> { using type = WarpBf16<D>; };
template <int D> struct WarpOf<float, D> { using type = WarpF32<D>; };

template <typename E, int D>
__global__ void __launch_bounds__(kWarps * 32) sink_decode_kernel(const __grid_constant__ DecodeArgs a) {
    using L = DecodeLayout<E, D>;
    extern __shared__ __align__(1024) unsigned char smem[];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Where w = where(a);
    const float scale_log2 = a.scale * 1.44269504088896340736f;
    char* kc = static_cast<char*>(a.kc) + w.kv_row * (a.n_sink + a.w) * L::ROW;
    char* vc = static_cast<char*>(a.vc) + w.kv_row * (a.n_sink + a.w) * L::ROW;
    const uint32_t ring = smem_u32(smem) + warp * L::STAGES * L::STAGE;
    const int stages = (w.n + kStageSlots - 1) / kStageSlots;
    const int first = w.rank * kWarps + warp, stride = w.split * kWarps;
    typename WarpOf<E, D>::type acc;
#pragma unroll
    for (int i = 0; i < L::STAGES - 1; ++i) {
        if (first + i * stride < stages) issue_stage<E, D>(ring + i * L::STAGE, kc, vc, first + i * stride, w.n, lane);
        cp_async_commit();
    }
    acc.init(a, w, lane);
    int buf = 0;
    for (int s = first; s < stages; s += stride) {
        const int ahead = s + (L::STAGES - 1) * stride;
        const int nbuf = buf == 0 ? L::STAGES - 1 : buf - 1;
        if (ahead < stages) issue_stage<E, D>(ring + nbuf * L::STAGE, kc, vc, ahead, w.n, lane);
        cp_async_commit();
        cp_async_wait<L::STAGES - 1>();
        __syncwarp();
        const uint32_t st = ring + buf * L::STAGE;
        if (w.slot / kStageSlots == s) put_token<E, D>(a, w, st, w.slot % kStageSlots, kc, vc, lane);
        acc.step(st, s * kStageSlots, w.n, scale_log2, lane);
        __syncwarp();                                        // the stage may be refilled
        buf = buf + 1 == L::STAGES ? 0 : buf + 1;
    }
    cp_async_wait<0>();
    __syncthreads();                                         // the ring becomes the accumulators' store
    float* accs = reinterpret_cast<float*>(smem);
    float* ml = reinterpret_cast<float*>(smem + L::OFF_ML);
    acc.store(accs + warp * kHeads * D, ml + warp * 2 * kHeads, lane);
    __syncthreads();
    // Join the warps: the block's accumulator over warp 0's, its (m, l) behind the warps'.
    float* bml = ml + kWarps * 2 * kHeads;
    for (int i = threadIdx.x; i < w.nh * D; i += kWarps * 32) {
        const int h = i / D;
        float mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) mx = fmaxf(mx, ml[k * 2 * kHeads + h]);
        const float mu = mx == -INFINITY ? 0.f : mx;
        float x = 0.f, sum = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
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
        for (int i = threadIdx.x; i < w.nh * D; i += kWarps * 32)
            y[i] = from_f32<E>(w.n > 0 ? accs[i] / bml[kHeads + i / D] : 0.f);
        return;
    }
    // Join the cluster's blocks: block `rank` writes its share of the outputs.
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    for (int i = w.rank * kWarps * 32 + threadIdx.x; i < w.nh * D; i += w.split * kWarps * 32) {
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

// Blocks per (sequence, key/value head, 16 heads): doubled while the blocks do not
// fill two per SM and each warp keeps at least 4 stages of a full window.
int plan_split(long long base, int slots, int num_sms) {
    int split = 1;
    while (split < kMaxSplit && base * split * 2 <= 2LL * num_sms && slots >= split * 2 * kWarps * kStageSlots * 4)
        split *= 2;
    return split;
}

template <typename E, int D>
cudaError_t run(DecodeArgs a, int B, int num_sms, cudaStream_t stream) {
    using L = DecodeLayout<E, D>;
    auto kern = sink_decode_kernel<E, D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    a.head_blocks = (a.Hq / a.Hkv + kHeads - 1) / kHeads;
    const long long base = (long long)B * a.Hkv * a.head_blocks;
    a.split = plan_split(base, a.n_sink + a.w, num_sms);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(base * a.split));
    cfg.blockDim = dim3(kWarps * 32);
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
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_sink_decode(void* k_cache, void* v_cache, const int64_t* positions, const void* q, const void* k,
                               const void* v, void* y, int B, int Hq, int Hkv, int d, int w, int n_sink, float scale,
                               bool bf16, int num_sms, unsigned* status, cudaStream_t stream) {
    (void)status;
    DecodeArgs a{k_cache, v_cache, positions, q, k, v, y, Hq, Hkv, w, n_sink, 1, 1, scale};
    if (bf16)
        return d == 64 ? run<__nv_bfloat16, 64>(a, B, num_sms, stream) : run<__nv_bfloat16, 128>(a, B, num_sms, stream);
    return d == 64 ? run<float, 64>(a, B, num_sms, stream) : run<float, 128>(a, B, num_sms, stream);
}

}  // namespace based
