// RMS norm of every query and key head with the rotation by position, forward and
// backward, each in one pass over memory.
//
//   n = x r weight, r = 1 / sqrt(mean(x^2) + eps); (a, b) -> (a c - b s, a s + b c)
// on the pairs of n's first `rot` channels. Backward, with dn the upstream
// gradient rotated back and xhat = x r:
//   dx = r (dn weight - xhat mean(dn weight xhat)),  dweight = sum dn xhat.
//
// A row (one head of one token) is held by LPR lanes, V + V channels each: the two
// pieces of a lane hold both members of its V pairs (channels p and p + rot/2 of the
// half-split order, 2 V neighbouring channels of the interleaved one and outside the
// rotated channels), so a rotation needs no exchange between lanes; only the sums of
// squares move by shuffles. A lane keeps one token and walks its heads, several at a
// time, so that the token's cos and sin are loaded once per walk and several rows are
// in flight per lane.
//
// Memory bounds it: 8 x 16+16 heads x 2048 x 64 bf16 move 139 MB in 28.4 us (4.9 TB/s, of
// 6.55 for a plain copy; 31.5 us with positions from memory, whose load the table's waits
// for), the gradient 206 MB in 52 us (4.0 TB/s, the sum of the weights' gradients
// included); one token of 64 sequences takes 2.4 us. fp32: 268 MB in 46 us (5.8 TB/s), the
// gradient 403 MB in 62 us (6.5 TB/s). Pieces of 16 bytes in the bf16
// forward: 30.0 -> 28.4 us, at d = 128 37.3 -> 33.0 (half the shuffles, loads and
// addresses per channel). The gradient keeps 4 channels a piece: it holds two rows and
// the weights' sums of both tensors in its registers.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace based {
namespace {

constexpr int kFwdThreads = 128, kFwdBlocksPerSm = 6;
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

// V channels as they are stored, and as pairs of floats.
template <typename T, int V> struct Piece;
template <> struct Piece<float, 4> {
    float4 v;
    __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void get(F2* x) const { x[0] = f2(v.x, v.y), x[1] = f2(v.z, v.w); }
    __device__ __forceinline__ void clear() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
};
__device__ __forceinline__ F2 unpack2(uint32_t w) { return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
template <> struct Piece<__nv_bfloat16, 4> {
    uint2 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void get(F2* x) const { x[0] = unpack2(v.x), x[1] = unpack2(v.y); }
    __device__ __forceinline__ void clear() { v = make_uint2(0u, 0u); }
};
template <> struct Piece<__nv_bfloat16, 8> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(F2* x) const {
        x[0] = unpack2(v.x), x[1] = unpack2(v.y), x[2] = unpack2(v.z), x[3] = unpack2(v.w);
    }
    __device__ __forceinline__ void clear() { v = make_uint4(0u, 0u, 0u, 0u); }
};
__device__ __forceinline__ uint32_t pack2(F2 x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(lo(x), hi(x));
    return *reinterpret_cast<const uint32_t*>(&a);
}
template <int V>
__device__ __forceinline__ void put(float* p, const F2* x) {
    *reinterpret_cast<float4*>(p) = make_float4(lo(x[0]), hi(x[0]), lo(x[1]), hi(x[1]));
}
template <int V>
__device__ __forceinline__ void put(__nv_bfloat16* p, const F2* x) {
    if constexpr (V == 4) *reinterpret_cast<uint2*>(p) = make_uint2(pack2(x[0]), pack2(x[1]));
    else *reinterpret_cast<uint4*>(p) = make_uint4(pack2(x[0]), pack2(x[1]), pack2(x[2]), pack2(x[3]));
}
// Rows in flight per lane (the gradient holds two tensors' rows).
constexpr int kFwdBatch = 2;
// Channels of a piece.
template <typename T> constexpr int kFwdPiece = sizeof(T) == 2 ? 8 : 4;
constexpr int kBwdPiece = 4;
template <typename T> constexpr int kBwdBatch = sizeof(T) == 2 ? 4 : 2;

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// What a lane keeps for its token: the place of its two pieces (channels ca.. and cb..)
// and the cos and sin of its V pairs.
template <int V, int LPR, bool INTERLEAVED>
struct Lane {
    int ca, cb;
    bool active, rotated;
    F2 c[V / 2], s[V / 2];                   // cos and sin, two pairs each

    __device__ __forceinline__ Lane(const RopeArgs& a) {
        const int lr = threadIdx.x % LPR;
        active = 2 * V * lr < a.d;
        rotated = 2 * V * lr < a.rot;
        const bool split = !INTERLEAVED && rotated;
        ca = split ? V * lr : 2 * V * lr;
        cb = split ? V * lr + a.rot / 2 : 2 * V * lr + V;
    }
    // Loads the token's cos and sin; false when its position is outside the table.
    __device__ __forceinline__ bool load(const RopeArgs& a, int b, int n) {
        if (a.rot == 0) return true;
        const long long pos = a.positions != nullptr ? a.positions[b * a.pos_sb + n] : n;
        if (pos < 0 || pos >= a.max_pos) return false;
        if (rotated) {                                       // pairs V lr .. of both orders
            const float4* t = reinterpret_cast<const float4*>(a.table + pos * a.rot + 2 * V * (threadIdx.x % LPR));
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float4 u = __ldg(t + i);
                c[i] = f2(u.x, u.z), s[i] = f2(u.y, u.w);
            }
        }
        return true;
    }
    // The weights of the lane's channels: piece a, then piece b.
    __device__ __forceinline__ void weights(const float* w, F2* out) const {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            float4 x = make_float4(1.f, 1.f, 1.f, 1.f);
            if (w != nullptr && active)
                x = __ldg(reinterpret_cast<const float4*>(w + (i < V / 4 ? ca + 4 * i : cb + 4 * i - V)));
            out[2 * i] = f2(x.x, x.y), out[2 * i + 1] = f2(x.z, x.w);
        }
    }
    // Rotates the lane's V + V channels by the angle (BACK: by minus the angle).
    template <bool BACK>
    __device__ __forceinline__ void rotate(F2* x) const {
        if (!rotated) return;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {                    // two pairs: first members a, second members b
            F2 &xa = INTERLEAVED ? x[2 * i] : x[i], &xb = INTERLEAVED ? x[2 * i + 1] : x[i + V / 2];
            F2 a = xa, b = xb;
            if (INTERLEAVED) a = f2(lo(xa), lo(xb)), b = f2(hi(xa), hi(xb));
            const F2 as = mul(a, s[i]), bs = mul(b, s[i]);
            a = fma(a, c[i], BACK ? bs : neg(bs));
            b = fma(b, c[i], BACK ? neg(as) : as);
            xa = INTERLEAVED ? f2(lo(a), lo(b)) : a;
            xb = INTERLEAVED ? f2(hi(a), hi(b)) : b;
        }
    }
};

template <int V, int LPR>
__device__ __forceinline__ float dot_row(const F2* x, const F2* y) {
    F2 t = mul(x[0], y[0]);
#pragma unroll
    for (int i = 1; i < V; ++i) t = fma(x[i], y[i], t);
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
    constexpr int kB = kFwdBatch, V = kFwdPiece<T>;
    grid_dependency_wait();
    grid_launch_dependents();
    Lane<V, LPR, INTERLEAVED> ln(a);
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
        F2 w[V];
        for (; h < hend; h += kB) {
            Piece<T, V> pa[kB], pb[kB];
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
                F2 x[V];
                pa[u].get(x);
                pb[u].get(x + V / 2);
                const float r = rsqrtf(dot_row<V, LPR>(x, x) * inv_d + a.eps) * poison;
                const F2 rr = f2(r, r);
#pragma unroll
                for (int i = 0; i < V; ++i) x[i] = mul(x[i], mul(rr, w[i]));
                ln.template rotate<false>(x);
                if (on) {
                    put<V>(dst + (h + u - hb) * out.sh + ln.ca, x);
                    put<V>(dst + (h + u - hb) * out.sh + ln.cb, x + V / 2);
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
    Lane<kBwdPiece, LPR, INTERLEAVED> ln(a);
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
                Piece<T, kBwdPiece> xa[kB], xb[kB], ga[kB], gb[kB];
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
                    const float r = rsqrtf(dot_row<kBwdPiece, LPR>(x, x) * inv_d + a.eps) * poison;
                    const F2 rr = f2(r, r);
                    ln.template rotate<true>(g);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[i] = mul(x[i], rr);                            // xhat
                        if (on) wsum[part][i] = fma(g[i], x[i], wsum[part][i]);
                        g[i] = mul(g[i], w[i]);
                    }
                    const float m = -dot_row<kBwdPiece, LPR>(g, x) * inv_d;
                    const F2 mm = f2(m, m);
#pragma unroll
                    for (int i = 0; i < 4; ++i) g[i] = mul(rr, fma(x[i], mm, g[i]));
                    if (on) {
                        put<kBwdPiece>(dst + (h + u - hb) * out.sh + ln.ca, g);
                        put<kBwdPiece>(dst + (h + u - hb) * out.sh + ln.cb, g + 2);
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

// Lanes of a row, `piece` + `piece` channels each.
int lanes_per_row(int d, int piece) {
    int l = 1;
    while (l * 2 * piece < d) l *= 2;
    return l;
}

// Heads per lane walk: up to 8, so that the table's cos and sin (from L2) cost
// little beside the rows, fewer when the tokens alone do not fill the SMs.
void plan_chunks(const RopeArgs& a, int lanes_row, int num_sms, int* chunks, int* per_chunk) {
    const int H = a.Hq + a.Hkv;
    const long long lanes = (long long)a.B * a.N * lanes_row;
    const long long want = ((long long)num_sms * 2048 + lanes - 1) / lanes;
    int c = (int)std::min<long long>(H, std::max<long long>((H + 7) / 8, want));
    *per_chunk = (H + c - 1) / c;
    *chunks = (H + *per_chunk - 1) / *per_chunk;
}

template <typename T, int LPR, bool INTERLEAVED, bool BACKWARD>
cudaError_t run(const RopeArgs& a, int num_sms, cudaStream_t stream) {
    int chunks, per_chunk;
    plan_chunks(a, LPR, num_sms, &chunks, &per_chunk);
    constexpr int tpb = (BACKWARD ? kBwdThreads : kFwdThreads) / LPR;
    const long long items = ((long long)a.B * a.N + tpb - 1) / tpb * chunks;
    if (items > 0x7fffffffLL) return cudaErrorInvalidValue;
    if constexpr (!BACKWARD) {
        return launch_pdl(rope_fwd_kernel<T, LPR, INTERLEAVED>, dim3((unsigned)items), dim3(kFwdThreads), 0, stream, a,
                          chunks, per_chunk);
    } else {
        const bool wgrad = a.dq_weight != nullptr || a.dk_weight != nullptr;
        float* partial = wgrad ? static_cast<float*>(a.workspace) : nullptr;
        const int blocks = (int)std::min<long long>(items, (long long)num_sms * kBwdBlocksPerSm);
        cudaError_t e = launch_pdl(rope_bwd_kernel<T, LPR, INTERLEAVED>, dim3(blocks), dim3(kBwdThreads), 0, stream, a,
                                   chunks, per_chunk, items, partial);
        if (e != cudaSuccess || !wgrad) return e;
        return launch_pdl(rope_weight_sum_kernel, dim3(2 * a.d / 32), dim3(1024), 0, stream,
                          static_cast<const float*>(partial), blocks, a.d, a.dq_weight, a.dk_weight);
    }
}

template <typename T, bool INTERLEAVED, bool BACKWARD>
cudaError_t pick(const RopeArgs& a, int num_sms, cudaStream_t stream) {
    constexpr int V = BACKWARD ? kBwdPiece : kFwdPiece<T>;
    switch (lanes_per_row(a.d, V)) {
        case 1:
            if constexpr (V == 8) return run<T, 1, INTERLEAVED, BACKWARD>(a, num_sms, stream);
            return cudaErrorInvalidValue;
        case 2: return run<T, 2, INTERLEAVED, BACKWARD>(a, num_sms, stream);
        case 4: return run<T, 4, INTERLEAVED, BACKWARD>(a, num_sms, stream);
        case 8: return run<T, 8, INTERLEAVED, BACKWARD>(a, num_sms, stream);
        case 16: return run<T, 16, INTERLEAVED, BACKWARD>(a, num_sms, stream);
        default:
            if constexpr (V == 4) return run<T, 32, INTERLEAVED, BACKWARD>(a, num_sms, stream);
            return cudaErrorInvalidValue;
    }
}

template <bool BACKWARD>
cudaError_t dispatch(const RopeArgs& a, bool bf16, int num_sms, cudaStream_t stream) {
    if (bf16)
        return a.interleaved ? pick<__nv_bfloat16, true, BACKWARD>(a, num_sms, stream)
                             : pick<__nv_bfloat16, false, BACKWARD>(a, num_sms, stream);
    return a.interleaved ? pick<float, true, BACKWARD>(a, num_sms, stream)
                         : pick<float, false, BACKWARD>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, bool bf16, int num_sms, cudaStream_t stream) {
    return dispatch<false>(a, bf16, num_sms, stream);
}

size_t qk_norm_rope_backward_workspace(int num_sms, int d) {
    return (size_t)num_sms * kBwdBlocksPerSm * 2 * d * sizeof(float);
}

cudaError_t launch_qk_norm_rope_backward(const RopeArgs& a, bool bf16, int num_sms, cudaStream_t stream) {
    return dispatch<true>(a, bf16, num_sms, stream);
}

cudaError_t launch_rope_table(float* table, int max_pos, int rot, double base, cudaStream_t stream) {
    const long long pairs = (long long)max_pos * (rot / 2);
    const int blocks = (int)std::min<long long>((pairs + 255) / 256, 4096);
    return launch_pdl(rope_table_kernel, dim3(blocks), dim3(256), 0, stream, reinterpret_cast<float2*>(table), pairs,
                      rot / 2, base);
}

}  // namespace based
