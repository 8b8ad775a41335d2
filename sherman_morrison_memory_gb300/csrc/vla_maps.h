// vla_maps.h -- tensor maps of strided sequences (host code).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace vla_layer {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

// Map of a bf16 sequence in boxes of 64 columns x `tokens` tokens; columns behind d
// and tokens behind T read as zero.
template <typename S>
inline bool make_map(CUtensorMap* m, const S* s, int B, int H, int T, int d, int tokens = 64) {
    const EncodeTiled fn = encode_tiled();
    if (!fn) return false;
    auto bytes = [](int n, long long st) { return (cuuint64_t)(n > 1 ? st * 2 : 16); };
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)T, (cuuint64_t)H, (cuuint64_t)B};
    const cuuint64_t strides[3] = {bytes(T, s->stride_t), bytes(H, s->stride_h), bytes(B, s->stride_b)};
    const cuuint32_t box[4] = {64, (cuuint32_t)tokens, 1, 1}, one[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, (void*)s->data, dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace vla_layer
