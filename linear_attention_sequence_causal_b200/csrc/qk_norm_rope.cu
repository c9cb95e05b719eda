// RMS norm of every query and key head with the rotation by position, forward and
// backward, each in one pass over memory.
//
//   n = x r weight, r = 1 / sqrt(mean(x^2) + eps); (a, b) -> (a c - b s, a s + b c)
// on the pairs of n's first `rot` channels. Backward, with dn the upstream
// gradient rotated back and xhat = x r:
//   dx = r (dn weight - xhat mean(dn weight xhat)),  dweight = sum dn xhat.
//
// A row (one head of one token) is held by LPR lanes, 4 + 4 channels each: the two
// pieces of a lane hold both members of its 4 pairs (channels p and p + rot/2 of the
// half-split order, 8 neighbouring channels of the interleaved one and outside the
// rotated channels), so a rotation needs no exchange between lanes; only the sums of
// squares move by shuffles. A lane keeps one token and walks its heads, several at a
// time, so that the token's cos and sin are loaded once per walk and several rows are
// in flight per lane. Memory bounds it.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace based {
namespace {

constexpr int kFwdThreads = 128, kFwdBlocksPerSm = 8;
constexpr int kBwdThreads = 256, kBwdBlocksPerSm = 2;

// Two fp32 operations in one instruction (the kernels issue near the SMs' rate).
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float lo(F2 x) { return __uint_as_float((uint32_t)x.v); }
__device__ __forceinline__ float hi(F2 x) { return __uint_as_float((uint32_t)(x.v >> 32)); }
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 neg(F2 a) { return f2(-lo(a), -hi(a)); }

// Four channels as they are stored, and as floats.
template <typename T> struct Piece;
template <> struct Piece<float> {
    float4 v;
    __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void get(F2* x) const { x[0] = f2(v.x, v.y), x[1] = f2(v.z, v.w); }
    __device__ __forceinline__ void clear() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
};
template <> struct Piece<__nv_bfloat16> {
    uint2 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void get(F2* x) const {
        x[0] = f2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u));
        x[1] = f2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
    }
    __device__ __forceinline__ void clear() { v = make_uint2(0u, 0u); }
};
__device__ __forceinline__ void store4(float* p, const F2* x) {
    *reinterpret_cast<float4*>(p) = make_float4(lo(x[0]), hi(x[0]), lo(x[1]), hi(x[1]));
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const F2* x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(lo(x[0]), hi(x[0])), b = __floats2bfloat162_rn(lo(x[1]), hi(x[1]));
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
// Rows in flight per lane (the gradient holds two tensors' rows).
template <typename T> constexpr int kFwdBatch = sizeof(T) == 2 ? 4 : 2;
template <typename T> constexpr int kBwdBatch = sizeof(T) == 2 ? 4 : 2;

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// What a lane keeps for its token: the place of its two pieces (channels ca.. and cb..)
// and the cos and sin of its four pairs.
template <int LPR, bool INTERLEAVED>
struct Lane {
    int ca, cb;
    bool active, rotated;
    F2 c[2], s[2];                           // cos and sin of pairs 0, 1 and 2, 3

    __device__ __forceinline__ Lane(const RopeArgs& a) {
        const int lr = threadIdx.x % LPR;
        active = 8 * lr < a.d;
        rotated = 8 * lr < a.rot;
        const bool split = !INTERLEAVED && rotated;
        ca = split ? 4 * lr : 8 * lr;
        cb = split ? 4 * lr + a.rot / 2 : 8 * lr + 4;
    }
    // Loads the token's cos and sin; false when its position is outside the table.
    __device__ __forceinline__ bool load(const RopeArgs& a, int b, int n) {
        if (a.rot == 0) return true;
        const long long pos = a.positions != nullptr ? a.positions[b * a.pos_sb + n] : n;
        if (pos < 0 || pos >= a.max_pos) return false;
        if (rotated) {                                       // pairs 4 lr .. of both orders
            const float4* t = reinterpret_cast<const float4*>(a.table + pos * a.rot + 8 * (threadIdx.x % LPR));
            const float4 u = __ldg(t), v = __ldg(t + 1);
            c[0] = f2(u.x, u.z), s[0] = f2(u.y, u.w);
            c[1] = f2(v.x, v.z), s[1] = f2(v.y, v.w);
        }
        return true;
    }
    // The weights of the lane's channels: out[0, 1] of piece a, out[2, 3] of piece b.
    __device__ __forceinline__ void weights(const float* w, F2* out) const {
        float4 a = make_float4(1.f, 1.f, 1.f, 1.f), b = a;
        if (w != nullptr && active) {
            a = __ldg(reinterpret_cast<const float4*>(w + ca));
            b = __ldg(reinterpret_cast<const float4*>(w + cb));
        }
        out[0] = f2(a.x, a.y), out[1] = f2(a.z, a.w), out[2] = f2(b.x, b.y), out[3] = f2(b.z, b.w);
    }
    // Rotates the lane's 4 + 4 channels by the angle (BACK: by minus the angle).
    template <bool BACK>
    __device__ __forceinline__ void rotate(F2* x) const {
        if (!rotated) return;
        F2 a[2] = {x[0], x[1]}, b[2] = {x[2], x[3]};         // first and second members of the pairs
        if (INTERLEAVED) {
            a[0] = f2(lo(x[0]), lo(x[1])), b[0] = f2(hi(x[0]), hi(x[1]));
            a[1] = f2(lo(x[2]), lo(x[3])), b[1] = f2(hi(x[2]), hi(x[3]));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const F2 as = mul(a[i], s[i]), bs = mul(b[i], s[i]);
            a[i] = fma(a[i], c[i], BACK ? bs : neg(bs));
            b[i] = fma(b[i], c[i], BACK ? neg(as) : as);
        }
        if (INTERLEAVED) {
            x[0] = f2(lo(a[0]), lo(b[0])), x[1] = f2(hi(a[0]), hi(b[0]));
            x[2] = f2(lo(a[1]), lo(b[1])), x[3] = f2(hi(a[1]), hi(b[1]));
        } else {
            x[0] = a[0], x[1] = a[1], x[2] = b[0], x[3] = b[1];
        }
    }
};

template <int LPR>
__device__ __forceinline__ float dot8(const F2* x, const F2* y) {
    F2 t = mul(x[0], y[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) t = fma(x[i], y[i], t);
    return row_sum<LPR>(lo(t) + hi(t));
}

// Work item -> (token of this lane, its heads [h0, h1)).
struct Item {
    int b, n, h0, h1;
    bool valid;
};
template <int THREADS, int LPR>
__device__ __forceinline__ Item item_of(const RopeArgs& a, long long it, int chunks, int per_chunk) {
    Item r;
    const long long tok = (it / chunks) * (THREADS / LPR) + threadIdx.x / LPR;
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
__global__ void __launch_bounds__(kFwdThreads, kFwdBlocksPerSm) rope_fwd_kernel(const __grid_constant__ RopeArgs a, int chunks,
                                                            int per_chunk) {
    constexpr int kB = kFwdBatch<T>;
    grid_dependency_wait();
    grid_launch_dependents();
    Lane<LPR, INTERLEAVED> ln(a);
    const Item it = item_of<kFwdThreads, LPR>(a, blockIdx.x, chunks, per_chunk);
    const bool on = it.valid && ln.active;
    const float inv_d = 1.0f / (float)a.d;
    float poison = 1.0f;
    bool ready = false;
    for (int h = it.h0; h < it.h1;) {
        const bool is_q = h < a.Hq;                          // uniform: a batch never mixes queries and keys
        const int hend = is_q ? min(it.h1, a.Hq) : it.h1;
        const View &in = is_q ? a.q : a.k, &out = is_q ? a.q_out : a.k_out;
        const int hb = is_q ? 0 : a.Hq;
        const T* src = static_cast<const T*>(in.p) + offset(in, it.b, 0, it.n);
        T* dst = static_cast<T*>(out.p) + offset(out, it.b, 0, it.n);
        F2 w[4];
        for (; h < hend; h += kB) {
            Piece<T> pa[kB], pb[kB];
#pragma unroll
            for (int u = 0; u < kB; ++u) {
                pa[u].clear();
                pb[u].clear();
                if (on && h + u < hend) {
                    pa[u].load(src + (h + u - hb) * in.sh + ln.ca);
                    pb[u].load(src + (h + u - hb) * in.sh + ln.cb);
                }
            }
            if (!ready) {                                    // behind the first rows' loads
                if (it.valid && !ln.load(a, it.b, it.n)) {
                    poison = __int_as_float(0x7fffffff);
                    atomicOr(a.status, DEV_ERR_RANGE);
                }
                ready = true;
            }
            ln.weights(is_q ? a.q_weight : a.k_weight, w);
#pragma unroll
            for (int u = 0; u < kB; ++u) {
                if (h + u >= hend) break;                    // uniform
                F2 x[4];
                pa[u].get(x);
                pb[u].get(x + 2);
                const float r = rsqrtf(dot8<LPR>(x, x) * inv_d + a.eps) * poison;
                const F2 rr = f2(r, r);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = mul(x[i], mul(rr, w[i]));
                ln.template rotate<false>(x);
                if (on) {
                    store4(dst + (h + u - hb) * out.sh + ln.ca, x);
                    store4(dst + (h + u - hb) * out.sh + ln.cb, x + 2);
                }
            }
        }
        h = hend;
    }
}

// Persistent: a block walks its items and keeps the weight gradients of its rows
// in registers; at the end it writes their sum to partial[block][q, k][d].
template <typename T, int LPR, bool INTERLEAVED>
__global__ void __launch_bounds__(kBwdThreads, kBwdBlocksPerSm) rope_bwd_kernel(const __grid_constant__ RopeArgs a, int chunks,
                                                            int per_chunk, long long items, float* partial) {
    constexpr int kB = kBwdBatch<T>;                         // rows in flight (x and the gradient of each)
    __shared__ float red[kBwdThreads / 32][2][LPR * 8];
    grid_dependency_wait();
    grid_launch_dependents();
    Lane<LPR, INTERLEAVED> ln(a);
    const float inv_d = 1.0f / (float)a.d;
    F2 wsum[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) wsum[0][i] = wsum[1][i] = f2(0.f, 0.f);
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
        const Item it = item_of<kBwdThreads, LPR>(a, item, chunks, per_chunk);
        const bool on = it.valid && ln.active;
        float poison = 1.0f;
        bool ready = false;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            const int hb = part == 0 ? 0 : a.Hq;
            const int h0 = max(it.h0, hb), hend = min(it.h1, part == 0 ? a.Hq : a.Hq + a.Hkv);
            if (h0 >= hend) continue;
            const View &in = part == 0 ? a.q : a.k, &up = part == 0 ? a.q_out : a.k_out,
                       &out = part == 0 ? a.dq : a.dk;
            const T* src = static_cast<const T*>(in.p) + offset(in, it.b, 0, it.n);
            const T* grd = static_cast<const T*>(up.p) + offset(up, it.b, 0, it.n);
            T* dst = static_cast<T*>(out.p) + offset(out, it.b, 0, it.n);
            F2 w[4];
            for (int h = h0; h < hend; h += kB) {
                Piece<T> xa[kB], xb[kB], ga[kB], gb[kB];
#pragma unroll
                for (int u = 0; u < kB; ++u) {
                    xa[u].clear(), xb[u].clear(), ga[u].clear(), gb[u].clear();
                    if (on && h + u < hend) {
                        xa[u].load(src + (h + u - hb) * in.sh + ln.ca);
                        xb[u].load(src + (h + u - hb) * in.sh + ln.cb);
                        ga[u].load(grd + (h + u - hb) * up.sh + ln.ca);
                        gb[u].load(grd + (h + u - hb) * up.sh + ln.cb);
                    }
                }
                if (!ready) {                                // behind the first rows' loads
                    if (it.valid && !ln.load(a, it.b, it.n)) {
                        poison = __int_as_float(0x7fffffff);
                        atomicOr(a.status, DEV_ERR_RANGE);
                    }
                    ready = true;
                }
                ln.weights(part == 0 ? a.q_weight : a.k_weight, w);
#pragma unroll
                for (int u = 0; u < kB; ++u) {
                    if (h + u >= hend) break;                // uniform
                    F2 x[4], g[4];
                    xa[u].get(x), xb[u].get(x + 2);
                    ga[u].get(g), gb[u].get(g + 2);
                    const float r = rsqrtf(dot8<LPR>(x, x) * inv_d + a.eps) * poison;
                    const F2 rr = f2(r, r);
                    ln.template rotate<true>(g);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[i] = mul(x[i], rr);                            // xhat
                        if (on) wsum[part][i] = fma(g[i], x[i], wsum[part][i]);
                        g[i] = mul(g[i], w[i]);
                    }
                    const float m = -dot8<LPR>(g, x) * inv_d;
                    const F2 mm = f2(m, m);
#pragma unroll
                    for (int i = 0; i < 4; ++i) g[i] = mul(rr, fma(x[i], mm, g[i]));
                    if (on) {
                        store4(dst + (h + u - hb) * out.sh + ln.ca, g);
                        store4(dst + (h + u - hb) * out.sh + ln.cb, g + 2);
                    }
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
            float s = i & 1 ? hi(wsum[part][i / 2]) : lo(wsum[part][i / 2]);
#pragma unroll
            for (int o = 16; o >= LPR; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane < LPR && ln.active) red[warp][part][i < 4 ? ln.ca + i : ln.cb + i - 4] = s;
        }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.d; c += kBwdThreads) {
        const int part = c / a.d, ch = c % a.d;
        float s = 0.f;
#pragma unroll
        for (int wp = 0; wp < kBwdThreads / 32; ++wp) s += red[wp][part][ch];
        partial[(size_t)blockIdx.x * 2 * a.d + c] = s;
    }
}

// dweight[c] = the sum of column c of partial [blocks][2 d]: 32 columns a block,
// the rows over its 32 warps, in a fixed order.
__global__ void __launch_bounds__(1024) rope_weight_sum_kernel(const float* partial, int blocks, int d, float* dq_weight,
                                                               float* dk_weight) {
    __shared__ float red[32][32];
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.f;
#pragma unroll 20
    for (int r = warp; r < blocks; r += 32) s += partial[(size_t)r * 2 * d + c];
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += red[i][lane];
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


template <typename T, int LPR, bool INTERLEAVED>
cudaError_t run(const RopeArgs& a, bool backward, int num_sms, cudaStream_t stream) {
    int chunks, per_chunk;
    plan_chunks(a, num_sms, &chunks, &per_chunk);
    const int threads = backward ? kBwdThreads : kFwdThreads, tpb = threads / LPR;
    const long long items = ((long long)a.B * a.N + tpb - 1) / tpb * chunks;
    if (items > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (!backward)
        return launch_pdl(rope_fwd_kernel<T, LPR, INTERLEAVED>, dim3((unsigned)items), dim3(kFwdThreads), 0, stream, a,
                          chunks, per_chunk);
    const bool wgrad = a.dq_weight != nullptr || a.dk_weight != nullptr;
    float* partial = wgrad ? static_cast<float*>(a.workspace) : nullptr;
    const int blocks = (int)std::min<long long>(items, (long long)num_sms * kBwdBlocksPerSm);
    cudaError_t e = launch_pdl(rope_bwd_kernel<T, LPR, INTERLEAVED>, dim3(blocks), dim3(kBwdThreads), 0, stream, a,
                               chunks, per_chunk, items, partial);
    if (e != cudaSuccess || !wgrad) return e;
    return launch_pdl(rope_weight_sum_kernel, dim3(2 * a.d / 32), dim3(1024), 0, stream,
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
