// Tensor maps of packed tokens' operands, for TMA copies.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace {

// A bf16 operand as a 3-D tensor of [tokens, heads or groups, columns] in boxes of `rows` tokens by
// 64 columns, 128-byte swizzle; false where the driver cannot describe it.
inline bool encode_map(CUtensorMap *map, const void *base, int64_t columns, int64_t heads,
                       int64_t tokens, int64_t head_stride, int64_t token_stride, int rows) {
    static const auto encode = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                             cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(fn);
    }();
    if (!encode) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(columns), static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(tokens)};
    // a dimension of one element has no stride of its own
    const cuuint64_t strides[2] = {
        static_cast<cuuint64_t>(heads > 1 ? head_stride * 2 : columns * 2),
        static_cast<cuuint64_t>(tokens > 1 ? token_stride * 2 : columns * heads * 2)};
    const cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(rows)}, steps[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims,
                  strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
