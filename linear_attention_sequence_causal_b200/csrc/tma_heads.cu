// Tensor maps of [B, H, N, d] views with strides of their own (see tma_host.cu for the lookup).
#include <mutex>

#include "tma_host.h"

namespace based {
namespace {

decltype(&cuTensorMapEncodeTiled) heads_encoder() {
    static decltype(&cuTensorMapEncodeTiled) fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<decltype(fn)>(p);
    });
    return fn;
}

}  // namespace

bool make_tmap_bf16_heads(CUtensorMap* map, const void* base, uint64_t x, uint64_t n, uint64_t h, uint64_t b,
                          uint64_t sn, uint64_t sh, uint64_t sb, uint32_t box_n) {
    const auto fn = heads_encoder();
    if (fn == nullptr) return false;
    const cuuint64_t dims[4] = {x, n, h, b};
    const cuuint64_t strides[3] = {sn * 2, sh * 2, sb * 2};    // bytes, dims 1 to 3
    const cuuint32_t box[4] = {64, box_n, 1, 1};
    const cuuint32_t estride[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estride,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace based
