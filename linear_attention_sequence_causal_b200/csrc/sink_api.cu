// C ABI of the sliding-window attention with sink tokens and of the query/key
// norm with rotation: argument validation and kernel selection. The contract of
// every entry point is in include/based.h.
#include <algorithm>
#include <cstdint>

#include "../../include/based.h"
#include "common.cuh"
#include "kernels.h"

namespace based {
unsigned* device_status_word(int dev);
int device_sm_count(int dev);
unsigned current_debug_flags();
}  // namespace based

namespace {

using based::View;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok_ptr(const void* p) { return p != nullptr && aligned16(p); }
bool ok_dtype(based_dtype_t d) { return d == BASED_F32 || d == BASED_BF16; }
bool is_finite(double x) { return x - x == 0.0; }

// Strides of one [B, H, N, d] tensor: the given ones (those of dimensions of size
// 1 replaced by what a dense tensor would have) or the dense ones. False when a
// stride is not a multiple of 16 bytes or two rows overlap. The bound on the
// total extent keeps every offset within 63 bits and within a tensor map.
bool make_view(View* out, const void* p, const based_strides_t* st, int B, int H, int N, int d, int esize) {
    if (!ok_ptr(p)) return false;
    out->p = const_cast<void*>(p);
    long long s[3] = {(long long)H * N * d, (long long)N * d, d};   // b, h, n
    if (st != nullptr) {
        const long long given[3] = {st->b, st->h, st->n}, size[3] = {B, H, N};
        // Dimensions larger than 1 in ascending order of stride must nest: each
        // stride covers the extent of all the smaller ones.
        int order[3], cnt = 0;
        for (int i = 0; i < 3; ++i)
            if (size[i] > 1) order[cnt++] = i;
        std::sort(order, order + cnt, [&](int a, int b) { return given[a] < given[b]; });
        long long extent = d;
        for (int i = 0; i < cnt; ++i) {
            const long long v = given[order[i]];
            if (v < extent || v % (16 / esize) != 0 || v > (1LL << 38) / size[order[i]]) return false;
            extent += v * (size[order[i]] - 1);
        }
        for (int i = 0; i < 3; ++i) s[i] = size[i] > 1 ? given[i] : (extent + 63) / 64 * 64;
    }
    out->sb = s[0];
    out->sh = s[1];
    out->sn = s[2];
    return true;
}

based_status_t device(int* dev, unsigned** status, int* sms) {
    if (cudaGetDevice(dev) != cudaSuccess) return BASED_ERR_CUDA;
    *status = based::device_status_word(*dev);
    *sms = based::device_sm_count(*dev);
    return (*status == nullptr || *sms <= 0) ? BASED_ERR_CUDA : BASED_OK;
}

// Sizes common to the attention calls.
based_status_t check_sizes(int B, int Hq, int Hkv, int N, int d, int w, int n_sink, float scale,
                           based_dtype_t dtype) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || N <= 0 || d <= 0 || w <= 0 || n_sink < 0 || !ok_dtype(dtype))
        return BASED_ERR_INVALID_ARG;
    if (Hq % Hkv != 0 || !(scale >= 0.0f) || !is_finite(scale)) return BASED_ERR_INVALID_ARG;
    if ((d != 64 && d != 128) || n_sink > based::kMaxSinks) return BASED_ERR_UNSUPPORTED;
    // Grid and index limits: 2^24 row tiles of 64, 2^29 tokens of window and of length
    // (so that a position plus a window stays within 31 bits).
    if (N > (1 << 29) || w > (1 << 29)) return BASED_ERR_UNSUPPORTED;
    if ((long long)B * Hq > (1LL << 24) || (long long)B * Hq * ((N + 63) / 64) > (1LL << 24))
        return BASED_ERR_UNSUPPORTED;
    if ((long long)B * Hq * N > (1LL << 38) / d) return BASED_ERR_UNSUPPORTED;
    return BASED_OK;
}

}  // namespace

extern "C" {

based_status_t based_swa_sink_prefill(const void* q, const based_strides_t* q_strides, const void* k,
                                      const based_strides_t* k_strides, const void* v,
                                      const based_strides_t* v_strides, void* y, const based_strides_t* y_strides,
                                      float* lse, void* k_cache, void* v_cache, const int64_t* lengths, int B, int Hq,
                                      int Hkv, int N, int d, int w, int n_sink, float scale, based_dtype_t dtype,
                                      cudaStream_t stream) {
    const based_status_t c = check_sizes(B, Hq, Hkv, N, d, w, n_sink, scale, dtype);
    if (c != BASED_OK) return c;
    const int es = dtype == BASED_BF16 ? 2 : 4;
    based::SinkArgs a{};
    if (!make_view(&a.q, q, q_strides, B, Hq, N, d, es) || !make_view(&a.k, k, k_strides, B, Hkv, N, d, es) ||
        !make_view(&a.v, v, v_strides, B, Hkv, N, d, es) || !make_view(&a.y, y, y_strides, B, Hq, N, d, es))
        return BASED_ERR_INVALID_ARG;
    if ((k_cache == nullptr) != (v_cache == nullptr) || !aligned16(lse) || !aligned16(k_cache) ||
        !aligned16(v_cache) || (reinterpret_cast<uintptr_t>(lengths) & 7u) != 0)
        return BASED_ERR_INVALID_ARG;
    if (k_cache != nullptr && (long long)B * Hkv * ((long long)w + n_sink) > (1LL << 38) / d)
        return BASED_ERR_UNSUPPORTED;
    int dev, sms;
    const based_status_t ds = device(&dev, &a.status, &sms);
    if (ds != BASED_OK) return ds;
    a.lse = lse;
    a.lengths = lengths;
    a.B = B, a.Hq = Hq, a.Hkv = Hkv, a.N = N, a.d = d, a.w = w, a.n_sink = n_sink;
    a.scale = scale;
    a.debug = based::current_debug_flags();
    a.fill = k_cache != nullptr;
    cudaError_t e = dtype == BASED_BF16 ? based::launch_sink_prefill_tc(a, sms, stream)
                                        : based::launch_sink_prefill_f32(a, stream);
    if (e == cudaSuccess && k_cache != nullptr)
        e = based::launch_sink_cache_fill(a, k_cache, v_cache, dtype == BASED_BF16, stream);
    return e == cudaSuccess ? BASED_OK : BASED_ERR_CUDA;
}

based_status_t based_swa_sink_decode(void* k_cache, void* v_cache, const int64_t* positions, const void* q,
                                     const void* k, const void* v, void* y, int B, int Hq, int Hkv, int d, int w,
                                     int n_sink, float scale, based_dtype_t dtype, cudaStream_t stream) {
    const based_status_t c = check_sizes(B, Hq, Hkv, 1, d, w, n_sink, scale, dtype);
    if (c != BASED_OK) return c;
    if (!ok_ptr(k_cache) || !ok_ptr(v_cache) || !ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(y) ||
        positions == nullptr || (reinterpret_cast<uintptr_t>(positions) & 7u) != 0)
        return BASED_ERR_INVALID_ARG;
    if ((long long)B * Hkv * ((long long)w + n_sink) > (1LL << 38) / d) return BASED_ERR_UNSUPPORTED;
    int dev, sms;
    unsigned* status;
    const based_status_t ds = device(&dev, &status, &sms);
    if (ds != BASED_OK) return ds;
    const cudaError_t e = based::launch_sink_decode(k_cache, v_cache, positions, q, k, v, y, B, Hq, Hkv, d, w, n_sink,
                                                    scale, dtype == BASED_BF16, sms, status, stream);
    return e == cudaSuccess ? BASED_OK : BASED_ERR_CUDA;
}

size_t based_swa_sink_backward_workspace(int B, int Hq, int Hkv, int N, int d, int w, int n_sink,
                                         based_dtype_t dtype) {
    if (check_sizes(B, Hq, Hkv, N, d, w, n_sink, 0.0f, dtype) != BASED_OK) return 0;
    return based::sink_backward_workspace(B, Hq, Hkv, N, d, w, n_sink, dtype == BASED_BF16);
}

based_status_t based_swa_sink_backward(
    const void* q, const based_strides_t* q_strides, const void* k, const based_strides_t* k_strides, const void* v,
    const based_strides_t* v_strides, const void* y, const based_strides_t* y_strides, const float* lse,
    const void* dy, const based_strides_t* dy_strides, void* dq, const based_strides_t* dq_strides, void* dk,
    const based_strides_t* dk_strides, void* dv, const based_strides_t* dv_strides, const int64_t* lengths, int B,
    int Hq, int Hkv, int N, int d, int w, int n_sink, float scale, based_dtype_t dtype, void* workspace,
    size_t workspace_bytes, cudaStream_t stream) {
    const based_status_t c = check_sizes(B, Hq, Hkv, N, d, w, n_sink, scale, dtype);
    if (c != BASED_OK) return c;
    const int es = dtype == BASED_BF16 ? 2 : 4;
    based::SinkArgs a{};
    if (!make_view(&a.q, q, q_strides, B, Hq, N, d, es) || !make_view(&a.k, k, k_strides, B, Hkv, N, d, es) ||
        !make_view(&a.v, v, v_strides, B, Hkv, N, d, es) || !make_view(&a.y, y, y_strides, B, Hq, N, d, es) ||
        !make_view(&a.dy, dy, dy_strides, B, Hq, N, d, es) || !make_view(&a.dq, dq, dq_strides, B, Hq, N, d, es) ||
        !make_view(&a.dk, dk, dk_strides, B, Hkv, N, d, es) || !make_view(&a.dv, dv, dv_strides, B, Hkv, N, d, es))
        return BASED_ERR_INVALID_ARG;
    if (!ok_ptr(lse) || (reinterpret_cast<uintptr_t>(lengths) & 7u) != 0) return BASED_ERR_INVALID_ARG;
    const size_t need = based::sink_backward_workspace(B, Hq, Hkv, N, d, w, n_sink, dtype == BASED_BF16);
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < need)
        return BASED_ERR_INVALID_ARG;
    int dev, sms;
    const based_status_t ds = device(&dev, &a.status, &sms);
    if (ds != BASED_OK) return ds;
    a.lse = const_cast<float*>(lse);
    a.lengths = lengths;
    a.B = B, a.Hq = Hq, a.Hkv = Hkv, a.N = N, a.d = d, a.w = w, a.n_sink = n_sink;
    a.scale = scale;
    a.workspace = workspace;
    a.debug = based::current_debug_flags();
    const cudaError_t e = dtype == BASED_BF16 ? based::launch_sink_backward_tc(a, sms, stream)
                                              : based::launch_sink_backward_f32(a, stream);
    return e == cudaSuccess ? BASED_OK : BASED_ERR_CUDA;
}

}  // extern "C"

namespace {

based_status_t check_rope(const float* q_weight, const float* k_weight, const float* table, int max_pos,
                          const int64_t* positions, int64_t pos_stride_b, int B, int Hq, int Hkv, int N, int d,
                          int rot, float eps, based_dtype_t dtype) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || N <= 0 || d <= 0 || rot < 0 || rot > d || !ok_dtype(dtype))
        return BASED_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !is_finite(eps)) return BASED_ERR_INVALID_ARG;
    if (!aligned16(q_weight) || !aligned16(k_weight)) return BASED_ERR_INVALID_ARG;
    if (rot > 0 && (!ok_ptr(table) || max_pos <= 0)) return BASED_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(positions) & 7u) != 0 ||
        (positions != nullptr && B > 1 && pos_stride_b != 0 && (pos_stride_b < N || pos_stride_b > (1LL << 38) / B)))
        return BASED_ERR_INVALID_ARG;
    if (d % 16 != 0 || d > 256 || rot % 16 != 0) return BASED_ERR_UNSUPPORTED;
    if ((long long)B * N > (1LL << 38) / ((long long)(Hq + Hkv) * d)) return BASED_ERR_UNSUPPORTED;
    return BASED_OK;
}

based::RopeArgs rope_args(const float* q_weight, const float* k_weight, const float* table, int max_pos,
                          const int64_t* positions, int64_t pos_stride_b, int B, int Hq, int Hkv, int N, int d,
                          int rot, int interleaved, float eps) {
    based::RopeArgs a{};
    a.q_weight = q_weight, a.k_weight = k_weight;
    a.table = table, a.max_pos = max_pos;
    a.positions = positions, a.pos_sb = pos_stride_b;
    a.B = B, a.Hq = Hq, a.Hkv = Hkv, a.N = N, a.d = d, a.rot = rot, a.interleaved = interleaved != 0;
    a.eps = eps;
    return a;
}

}  // namespace

extern "C" {

based_status_t based_qk_norm_rope(const void* q, const based_strides_t* q_strides, const void* k,
                                  const based_strides_t* k_strides, void* q_out,
                                  const based_strides_t* q_out_strides, void* k_out,
                                  const based_strides_t* k_out_strides, const float* q_weight, const float* k_weight,
                                  const float* table, int max_pos, const int64_t* positions, int64_t pos_stride_b,
                                  int B, int Hq, int Hkv, int N, int d, int rot, int interleaved, float eps,
                                  based_dtype_t dtype, cudaStream_t stream) {
    const based_status_t c = check_rope(q_weight, k_weight, table, max_pos, positions, pos_stride_b, B, Hq, Hkv, N, d,
                                        rot, eps, dtype);
    if (c != BASED_OK) return c;
    const int es = dtype == BASED_BF16 ? 2 : 4;
    based::RopeArgs a = rope_args(q_weight, k_weight, table, max_pos, positions, pos_stride_b, B, Hq, Hkv, N, d, rot,
                                  interleaved, eps);
    if (!make_view(&a.q, q, q_strides, B, Hq, N, d, es) || !make_view(&a.k, k, k_strides, B, Hkv, N, d, es) ||
        !make_view(&a.q_out, q_out, q_out_strides, B, Hq, N, d, es) ||
        !make_view(&a.k_out, k_out, k_out_strides, B, Hkv, N, d, es))
        return BASED_ERR_INVALID_ARG;
    int dev, sms;
    const based_status_t ds = device(&dev, &a.status, &sms);
    if (ds != BASED_OK) return ds;
    const cudaError_t e = based::launch_qk_norm_rope(a, dtype == BASED_BF16, sms, stream);
    return e == cudaSuccess ? BASED_OK : BASED_ERR_CUDA;
}

size_t based_qk_norm_rope_backward_workspace(int B, int Hq, int Hkv, int N, int d, based_dtype_t dtype) {
    if (check_rope(nullptr, nullptr, nullptr, 0, nullptr, 0, B, Hq, Hkv, N, d, 0, 0.0f, dtype) != BASED_OK) return 0;
    int dev;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const int sms = based::device_sm_count(dev);
    return sms > 0 ? based::qk_norm_rope_backward_workspace(sms, d) : 0;
}

based_status_t based_qk_norm_rope_backward(
    const void* q, const based_strides_t* q_strides, const void* k, const based_strides_t* k_strides,
    const void* dq_out, const based_strides_t* dq_out_strides, const void* dk_out,
    const based_strides_t* dk_out_strides, void* dq, const based_strides_t* dq_strides, void* dk,
    const based_strides_t* dk_strides, float* dq_weight, float* dk_weight, const float* q_weight,
    const float* k_weight, const float* table, int max_pos, const int64_t* positions, int64_t pos_stride_b, int B,
    int Hq, int Hkv, int N, int d, int rot, int interleaved, float eps, based_dtype_t dtype, void* workspace,
    size_t workspace_bytes, cudaStream_t stream) {
    const based_status_t c = check_rope(q_weight, k_weight, table, max_pos, positions, pos_stride_b, B, Hq, Hkv, N, d,
                                        rot, eps, dtype);
    if (c != BASED_OK) return c;
    const int es = dtype == BASED_BF16 ? 2 : 4;
    based::RopeArgs a = rope_args(q_weight, k_weight, table, max_pos, positions, pos_stride_b, B, Hq, Hkv, N, d, rot,
                                  interleaved, eps);
    if (!make_view(&a.q, q, q_strides, B, Hq, N, d, es) || !make_view(&a.k, k, k_strides, B, Hkv, N, d, es) ||
        !make_view(&a.q_out, dq_out, dq_out_strides, B, Hq, N, d, es) ||
        !make_view(&a.k_out, dk_out, dk_out_strides, B, Hkv, N, d, es) ||
        !make_view(&a.dq, dq, dq_strides, B, Hq, N, d, es) || !make_view(&a.dk, dk, dk_strides, B, Hkv, N, d, es))
        return BASED_ERR_INVALID_ARG;
    if (!aligned16(dq_weight) || !aligned16(dk_weight) || !aligned16(workspace)) return BASED_ERR_INVALID_ARG;
    int dev, sms;
    const based_status_t ds = device(&dev, &a.status, &sms);
    if (ds != BASED_OK) return ds;
    if ((dq_weight != nullptr || dk_weight != nullptr) &&
        (workspace == nullptr || workspace_bytes < based::qk_norm_rope_backward_workspace(sms, d)))
        return BASED_ERR_INVALID_ARG;
    a.dq_weight = dq_weight, a.dk_weight = dk_weight;
    a.workspace = workspace;
    const cudaError_t e = based::launch_qk_norm_rope_backward(a, dtype == BASED_BF16, sms, stream);
    return e == cudaSuccess ? BASED_OK : BASED_ERR_CUDA;
}

based_status_t based_rope_table(float* table, int max_pos, int rot, double base, cudaStream_t stream) {
    if (!ok_ptr(table) || max_pos <= 0 || rot <= 0 || !(base > 0.0) || !is_finite(base)) return BASED_ERR_INVALID_ARG;
    if (rot % 16 != 0 || rot > 256) return BASED_ERR_UNSUPPORTED;
    return based::launch_rope_table(table, max_pos, rot, base, stream) == cudaSuccess ? BASED_OK : BASED_ERR_CUDA;
}

}  // extern "C"
