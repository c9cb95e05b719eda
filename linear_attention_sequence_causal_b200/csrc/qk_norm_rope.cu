// RMS norm of every query and key head with the rotation by position, forward and
// backward, each in one pass over memory.
//
//   n = x r weight, r = 1 / sqrt(mean(x^2) + eps); (a, b) -> (a c - b s, a s + b c)
// on the pairs of n's first `rot` channels. Backward, with dn the upstream
// gradient rotated back and xhat = x r:
//   dx = r (dn weight - xhat mean(dn weight xhat)),  dweight = sum dn xhat.
//
// A row (one head of one token) is held by LPR lanes, 8 channels each, so both
// sums of squares and the partner channels of the half-split pairs move by
// shuffles and nothing is staged. A lane keeps one token and walks its heads, 4 at
// a time, so that the token's cos and sin are loaded once per walk and 4 rows are
// in flight per lane. Memory bounds it: B=8, N=2048, 16+16 heads of 64, bf16.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace based {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;                // rows in flight per lane

__device__ __forceinline__ void load8(const float* p, float* x) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Rotates one row by its cos and sin (cs: pairs of this lane's channels); `sign`
// -1 rotates back. src is the lane that holds this lane's partner channels of the
// half-split pairs (its own lane outside the rotated channels); `first` says that
// this lane holds the pairs' first members.
template <bool INTERLEAVED>
__device__ __forceinline__ void rotate(float* x, const float* cs, float sign, bool rotated, bool first, int src) {
    if constexpr (INTERLEAVED) {
        if (rotated) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float c = cs[2 * i], s = sign * cs[2 * i + 1];
                const float a = x[2 * i], b = x[2 * i + 1];
                x[2 * i] = a * c - b * s;
                x[2 * i + 1] = a * s + b * c;
            }
        }
    } else {
        const float sg = first ? -sign : sign;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p = __shfl_sync(0xffffffffu, x[i], src);
            if (rotated) x[i] = x[i] * cs[2 * i] + p * (sg * cs[2 * i + 1]);
        }
    }
}

// What a lane keeps for its token: channel role and the token's cos and sin.
template <int LPR, bool INTERLEAVED>
struct Lane {
    int lr, c0, src;
    bool active, rotated, first;
    float cs[INTERLEAVED ? 8 : 16];

    __device__ __forceinline__ Lane(const RopeArgs& a) {
        const int lane = threadIdx.x & 31;
        lr = threadIdx.x % LPR;
        c0 = 8 * lr;
        active = c0 < a.d;
        rotated = c0 < a.rot;
        first = c0 < a.rot / 2;
        src = !rotated ? lane : first ? lane + a.rot / 16 : lane - a.rot / 16;
    }
    // Loads the token's cos and sin; false when its position is outside the table.
    __device__ __forceinline__ bool load(const RopeArgs& a, int b, int n) {
        if (a.rot == 0) return true;
        const long long pos = a.positions != nullptr ? a.positions[b * a.pos_sb + n] : n;
        if (pos < 0 || pos >= a.max_pos) return false;
        if (rotated) {
            const int pair = INTERLEAVED ? c0 / 2 : (first ? c0 : c0 - a.rot / 2);
            const float4* t = reinterpret_cast<const float4*>(a.table + pos * a.rot + 2 * pair);
#pragma unroll
            for (int i = 0; i < (INTERLEAVED ? 2 : 4); ++i) {
                const float4 v = __ldg(t + i);
                cs[4 * i] = v.x, cs[4 * i + 1] = v.y, cs[4 * i + 2] = v.z, cs[4 * i + 3] = v.w;
            }
        }
        return true;
    }
    __device__ __forceinline__ void weights(const float* w, float* out) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = (w != nullptr && active) ? __ldg(w + c0 + i) : 1.0f;
    }
};

// Work item -> (token of this lane, its heads [h0, h1)).
struct Item {
    int b, n, h0, h1;
    bool valid;
};
template <int LPR>
__device__ __forceinline__ Item item_of(const RopeArgs& a, long long it, int chunks, int per_chunk) {
    Item r;
    const long long tok = (it / chunks) * (kThreads / LPR) + threadIdx.x / LPR;
    r.valid = tok < (long long)a.B * a.N;
    r.b = r.valid ? (int)(tok / a.N) : 0;
    r.n = r.valid ? (int)(tok % a.N) : 0;
    r.h0 = (int)(it % chunks) * per_chunk;
    r.h1 = min(a.Hq + a.Hkv, r.h0 + per_chunk);
    return r;
}

// Element offset of head h (queries first, then keys) of token (b, n).
__device__ __forceinline__ size_t offset(const View& v, int b, int h, int n) {
    return (size_t)(b * v.sb + h * v.sh + n * v.sn);
}

template <typename T, int LPR, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rope_fwd_kernel(const __grid_constant__ RopeArgs a, int chunks,
                                                            int per_chunk) {
    grid_dependency_wait();
    grid_launch_dependents();
    Lane<LPR, INTERLEAVED> ln(a);
    const Item it = item_of<LPR>(a, blockIdx.x, chunks, per_chunk);
    const float nan = __int_as_float(0x7fffffff);
    float poison = 1.0f;
    if (it.valid && !ln.load(a, it.b, it.n)) {
        poison = nan;
        atomicOr(a.status, DEV_ERR_RANGE);
    }
    const float inv_d = 1.0f / (float)a.d;
    for (int h = it.h0; h < it.h1;) {
        const bool is_q = h < a.Hq;                          // uniform: a batch never mixes queries and keys
        const int hend = is_q ? min(it.h1, a.Hq) : it.h1;
        const View &in = is_q ? a.q : a.k, &out = is_q ? a.q_out : a.k_out;
        const int hb = is_q ? 0 : a.Hq;
        float w[8];
        ln.weights(is_q ? a.q_weight : a.k_weight, w);
        for (; h < hend; h += kBatch) {
            float x[kBatch][8];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[u][i] = 0.f;
                if (it.valid && ln.active && h + u < hend)
                    load8(static_cast<const T*>(in.p) + offset(in, it.b, h + u - hb, it.n) + ln.c0, x[u]);
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[u][i], x[u][i], ss);
                const float r = rsqrtf(row_sum<LPR>(ss) * inv_d + a.eps) * poison;
#pragma unroll
                for (int i = 0; i < 8; ++i) x[u][i] *= r * w[i];
                rotate<INTERLEAVED>(x[u], ln.cs, 1.0f, ln.rotated, ln.first, ln.src);
                if (it.valid && ln.active && h + u < hend)
                    store8(static_cast<T*>(out.p) + offset(out, it.b, h + u - hb, it.n) + ln.c0, x[u]);
            }
        }
        h = hend;
    }
}

// Persistent: a block walks its items and keeps the weight gradients of its rows
// in registers; at the end it writes their sum to partial[block][q, k][d].
template <typename T, int LPR, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rope_bwd_kernel(const __grid_constant__ RopeArgs a, int chunks,
                                                            int per_chunk, long long items, float* partial) {
    constexpr int kB = 2;                                    // rows in flight (x and the gradient of each)
    __shared__ float red[kThreads / 32][2][LPR * 8];
    grid_dependency_wait();
    grid_launch_dependents();
    Lane<LPR, INTERLEAVED> ln(a);
    const float nan = __int_as_float(0x7fffffff);
    const float inv_d = 1.0f / (float)a.d;
    float wsum[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) wsum[0][i] = wsum[1][i] = 0.f;
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
        const Item it = item_of<LPR>(a, item, chunks, per_chunk);
        float poison = 1.0f;
        if (it.valid && !ln.load(a, it.b, it.n)) {
            poison = nan;
            atomicOr(a.status, DEV_ERR_RANGE);
        }
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            const int hb = part == 0 ? 0 : a.Hq;
            const int h0 = max(it.h0, hb), hend = min(it.h1, part == 0 ? a.Hq : a.Hq + a.Hkv);
            if (h0 >= hend) continue;
            const View &in = part == 0 ? a.q : a.k, &up = part == 0 ? a.q_out : a.k_out,
                       &out = part == 0 ? a.dq : a.dk;
            float w[8];
            ln.weights(part == 0 ? a.q_weight : a.k_weight, w);
            for (int h = h0; h < hend; h += kB) {
                float x[kB][8], g[kB][8];
#pragma unroll
                for (int u = 0; u < kB; ++u) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[u][i] = g[u][i] = 0.f;
                    if (it.valid && ln.active && h + u < hend) {
                        load8(static_cast<const T*>(in.p) + offset(in, it.b, h + u - hb, it.n) + ln.c0, x[u]);
                        load8(static_cast<const T*>(up.p) + offset(up, it.b, h + u - hb, it.n) + ln.c0, g[u]);
                    }
                }
#pragma unroll
                for (int u = 0; u < kB; ++u) {
                    const bool live = it.valid && ln.active && h + u < hend;
                    float ss = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss = fmaf(x[u][i], x[u][i], ss);
                    const float r = rsqrtf(row_sum<LPR>(ss) * inv_d + a.eps) * poison;
                    rotate<INTERLEAVED>(g[u], ln.cs, -1.0f, ln.rotated, ln.first, ln.src);
                    float dot = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[u][i] *= r;                                    // xhat
                        if (live) wsum[part][i] = fmaf(g[u][i], x[u][i], wsum[part][i]);
                        g[u][i] *= w[i];
                        dot = fmaf(g[u][i], x[u][i], dot);
                    }
                    const float m = row_sum<LPR>(dot) * inv_d;
#pragma unroll
                    for (int i = 0; i < 8; ++i) g[u][i] = r * (g[u][i] - x[u][i] * m);
                    if (live)
                        store8(static_cast<T*>(out.p) + offset(out, it.b, h + u - hb, it.n) + ln.c0, g[u]);
                }
            }
        }
    }
    if (partial == nullptr) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float s = wsum[part][i];
#pragma unroll
            for (int o = 16; o >= LPR; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane < LPR) red[warp][part][8 * lane + i] = s;
        }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.d; c += kThreads) {
        const int part = c / a.d, ch = c % a.d;
        float s = 0.f;
#pragma unroll
        for (int wp = 0; wp < kThreads / 32; ++wp) s += red[wp][part][ch];
        partial[(size_t)blockIdx.x * 2 * a.d + c] = s;
    }
}

// dweight[c] = the sum of column c of partial [blocks][2 d]: 32 columns a block,
// the rows over its 8 warps, in a fixed order.
__global__ void __launch_bounds__(256) rope_weight_sum_kernel(const float* partial, int blocks, int d, float* dq_weight,
                                                              float* dk_weight) {
    __shared__ float red[8][32];
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.f;
#pragma unroll 8
    for (int r = warp; r < blocks; r += 8) s += partial[(size_t)r * 2 * d + c];
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += red[i][lane];
        float* out = c < d ? dq_weight : dk_weight;
        if (out != nullptr) out[c < d ? c : c - d] = t;
    }
}

__global__ void __launch_bounds__(256) rope_table_kernel(float2* table, long long pairs, int half, double base) {
    grid_dependency_wait();
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < pairs; i += (long long)gridDim.x * 256) {
        const double f = pow(base, -(double)(i % half) / (double)half);   // 2 i / rot = i / half
        double s, c;
        sincos((double)(i / half) * f, &s, &c);
        table[i] = make_float2((float)c, (float)s);
    }
}

int lanes_per_row(int d) {
    int l = 2;
    while (l * 8 < d) l *= 2;
    return l;
}

// Heads per lane walk: up to 8, so that the table's cos and sin (from L2) cost
// little beside the rows, fewer when the tokens alone do not fill the SMs.
void plan_chunks(const RopeArgs& a, int num_sms, int* chunks, int* per_chunk) {
    const int H = a.Hq + a.Hkv;
    const long long lanes = (long long)a.B * a.N * lanes_per_row(a.d);
    const long long want = ((long long)num_sms * 2048 + lanes - 1) / lanes;
    int c = (int)std::min<long long>(H, std::max<long long>((H + 7) / 8, want));
    *per_chunk = (H + c - 1) / c;
    *chunks = (H + *per_chunk - 1) / *per_chunk;
}

constexpr int kBwdBlocksPerSm = 4;

template <typename T, int LPR, bool INTERLEAVED>
cudaError_t run(const RopeArgs& a, bool backward, int num_sms, cudaStream_t stream) {
    int chunks, per_chunk;
    plan_chunks(a, num_sms, &chunks, &per_chunk);
    const int tpb = kThreads / LPR;
    const long long items = ((long long)a.B * a.N + tpb - 1) / tpb * chunks;
    if (items > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (!backward)
        return launch_pdl(rope_fwd_kernel<T, LPR, INTERLEAVED>, dim3((unsigned)items), dim3(kThreads), 0, stream, a,
                          chunks, per_chunk);
    const bool wgrad = a.dq_weight != nullptr || a.dk_weight != nullptr;
    float* partial = wgrad ? static_cast<float*>(a.workspace) : nullptr;
    const int blocks = (int)std::min<long long>(items, (long long)num_sms * kBwdBlocksPerSm);
    cudaError_t e = launch_pdl(rope_bwd_kernel<T, LPR, INTERLEAVED>, dim3(blocks), dim3(kThreads), 0, stream, a,
                               chunks, per_chunk, items, partial);
    if (e != cudaSuccess || !wgrad) return e;
    return launch_pdl(rope_weight_sum_kernel, dim3(2 * a.d / 32), dim3(256), 0, stream,
                      static_cast<const float*>(partial), blocks, a.d, a.dq_weight, a.dk_weight);
}

template <typename T, bool INTERLEAVED>
cudaError_t pick(const RopeArgs& a, bool backward, int num_sms, cudaStream_t stream) {
    switch (lanes_per_row(a.d)) {
        case 2: return run<T, 2, INTERLEAVED>(a, backward, num_sms, stream);
        case 4: return run<T, 4, INTERLEAVED>(a, backward, num_sms, stream);
        case 8: return run<T, 8, INTERLEAVED>(a, backward, num_sms, stream);
        case 16: return run<T, 16, INTERLEAVED>(a, backward, num_sms, stream);
        default: return run<T, 32, INTERLEAVED>(a, backward, num_sms, stream);
    }
}

cudaError_t dispatch(const RopeArgs& a, bool bf16, bool backward, int num_sms, cudaStream_t stream) {
    if (bf16)
        return a.interleaved ? pick<__nv_bfloat16, true>(a, backward, num_sms, stream)
                             : pick<__nv_bfloat16, false>(a, backward, num_sms, stream);
    return a.interleaved ? pick<float, true>(a, backward, num_sms, stream)
                         : pick<float, false>(a, backward, num_sms, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, bool bf16, int num_sms, cudaStream_t stream) {
    return dispatch(a, bf16, false, num_sms, stream);
}

size_t qk_norm_rope_backward_workspace(int num_sms, int d) {
    return (size_t)num_sms * kBwdBlocksPerSm * 2 * d * sizeof(float);
}

cudaError_t launch_qk_norm_rope_backward(const RopeArgs& a, bool bf16, int num_sms, cudaStream_t stream) {
    return dispatch(a, bf16, true, num_sms, stream);
}

cudaError_t launch_rope_table(float* table, int max_pos, int rot, double base, cudaStream_t stream) {
    const long long pairs = (long long)max_pos * (rot / 2);
    const int blocks = (int)std::min<long long>((pairs + 255) / 256, 4096);
    return launch_pdl(rope_table_kernel, dim3(blocks), dim3(256), 0, stream, reinterpret_cast<float2*>(table), pairs,
                      rot / 2, base);
}

}  // namespace based
