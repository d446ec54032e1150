// stq_map.h -- tensor maps of token rows, for TMA loads.
#pragma once

#include <cuda.h>

#include "stq_internal.h"

namespace stq {

// cuTensorMapEncodeTiled, from the driver that the runtime has loaded.
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled()
{
    static const EncodeTiled f = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

// Rows [tokens][heads][128] in boxes of 64 dims x `box_heads` heads x `box_tokens` tokens.
inline bool make_map(CUtensorMap *map, const stq_rows &r, int32_t dtype, int tokens, int heads, int box_heads, int box_tokens)
{
    const EncodeTiled encode = encode_tiled();
    if (encode == nullptr) return false;
    // a dimension of one element has no stride; the map wants some valid one
    const cuuint64_t dims[3] = {kD, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(heads > 1 ? r.head_stride : kD) * 2,
                                   static_cast<cuuint64_t>(tokens > 1 ? r.token_stride : kD) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_tokens)};
    const cuuint32_t step[3] = {1, 1, 1};
    return encode(map, dtype == STQ_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                  const_cast<void *>(r.data), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether a map can describe the rows: it takes positive strides only.
inline bool rows_mappable(const stq_rows &r, int heads, int tokens)
{
    const int64_t most = int64_t(1) << 38;
    return (heads <= 1 || (r.head_stride > 0 && r.head_stride < most)) && (tokens <= 1 || (r.token_stride > 0 && r.token_stride < most));
}

}  // namespace stq
