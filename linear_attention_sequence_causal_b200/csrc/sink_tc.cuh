// Device helpers shared by the tensor-core kernels of the sink-window attention.
#pragma once

#include "sink.cuh"
#include "tcgen05_heads.cuh"
#include "tma_host.h"

namespace based {
namespace tc {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// (a, b) = (x, y) c + d with the packed fp32 FMA.
__device__ __forceinline__ void scale_pair(float x, float y, float c, float d, float& a, float& b) {
    asm("{\n\t.reg .b64 x, c, d;\n\t"
        "mov.b64 x, {%2, %3};\n\t"
        "mov.b64 c, {%4, %4};\n\t"
        "mov.b64 d, {%5, %5};\n\t"
        "fma.rn.f32x2 x, x, c, d;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "=f"(a), "=f"(b)
        : "f"(x), "f"(y), "f"(c), "f"(d));
}

// The weights of 32 columns: p = 2^(s c - m), packed to bf16 (the product's operand type:
// at most 2^-8 of a weight, independent from one to the next); l0, l1 += the unrounded
// weights. One loop per operation: written pair by pair, each pair waits out its own
// exponentials (551 cycles against 320 for one warp, which is near the 256 that 32
// exponentials take).
__device__ __forceinline__ void weights32(float* s, float c, float m, uint32_t* out, float& l0, float& l1) {
#pragma unroll
    for (int i = 0; i < 16; ++i) scale_pair(s[2 * i], s[2 * i + 1], c, -m, s[2 * i], s[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < 32; ++i) s[i] = ex2(s[i]);
    float k0 = 0.f, k1 = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        add_pair(l0, l1, s[2 * i], s[2 * i + 1]);
        add_pair(k0, k1, s[2 * i + 2], s[2 * i + 3]);
    }
    add_pair(l0, l1, k0, k1);
#pragma unroll
    for (int i = 0; i < 16; ++i) out[i] = pack_bf16x2(s[2 * i], s[2 * i + 1]);
}

// mbar_wait by a whole warp whose lanes go on or give up together: in a wait that runs out as
// its phase completes, some could do either, and the warp's next joint instruction would wait
// for the ones that left.
__device__ __forceinline__ bool mbar_wait_joint(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned* status) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status));
}

// The n lowest bits (none below 0, all from 32 on).
__device__ __forceinline__ uint32_t low_bits(int n) {
    return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
}

// The visible columns of one 32-column word, and whether the rows of the warp see all or
// none of it. (Tests of bounds in place of bits, picked by more votes, were slower: the
// bit tests compile to one predicate load per seven scores.)
struct WordMask {
    enum Kind { kAll, kNone, kBits };
    uint32_t bits;
    int kind;

    __device__ __forceinline__ explicit WordMask(uint32_t vis) : bits(vis) {
        kind = __all_sync(0xffffffffu, vis == ~0u) ? kAll : __any_sync(0xffffffffu, vis != 0u) ? kBits : kNone;
    }
    // x where visible, else `hidden`.
    __device__ __forceinline__ void apply(float* x, float hidden) const {
        if (kind == kBits) {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = (bits & (1u << i)) != 0u ? x[i] : hidden;
        }
    }
};

__device__ __forceinline__ float max32(const float* s) {
    float m[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int q = 4; q < 28; q += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], fmaxf(s[q + 2 * e], s[q + 2 * e + 1]));
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], s[28 + e]);
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// Multiplies `n` columns of this thread's row of an accumulator.
template <int N>
__device__ __forceinline__ void scale_row(uint32_t taddr, float f) {
#pragma unroll
    for (int q = 0; q < N / 16; ++q) {
        float o[16];
        uint32_t ob[16];
        tmem_ld16(taddr + 16 * q, o);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) ob[e] = __float_as_uint(o[e] * f);
        tmem_st16(taddr + 16 * q, ob);
    }
}

}  // namespace tc

// Tensor map of a [B, H, N, d] view in tiles of 64 channels x `rows` tokens.
inline bool heads_map(CUtensorMap* m, const View& v, const SinkArgs& a, int H, uint32_t rows) {
    return make_tmap_bf16_heads(m, v.p, a.d, a.N, H, a.B, v.sn, v.sh, v.sb, rows);
}

}  // namespace based
