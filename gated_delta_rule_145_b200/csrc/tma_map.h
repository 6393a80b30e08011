// tma_map.h -- host-side construction of 2-D bf16 TMA tensor maps [rows, width]: the
// tensor-core prefill's (boxes of 64 elements x 32 rows with the 128-byte swizzle, one box
// row = one 128-byte swizzle row) and plain row-major boxes for streaming passes.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gdr {

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }
    return fn;
}

// Row pitch = width elements (16-byte multiple); rows outside [0, rows) read as zero.
inline bool make_bf16_map(CUtensorMap* map, const void* base, uint64_t width, uint64_t rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {width, rows};
    const cuuint64_t strides[1] = {width * 2};
    const cuuint32_t box[2] = {64, 32};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
               box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// Row pitch = width elements (16-byte multiple); boxes of box_w x box_h elements stored
// row-major without swizzle; rows and columns outside the tensor read as zero.
inline bool make_bf16_map_plain(CUtensorMap* map, const void* base, uint64_t width,
                                uint64_t rows, uint32_t box_w, uint32_t box_h) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {width, rows};
    const cuuint64_t strides[1] = {width * 2};
    const cuuint32_t box[2] = {box_w, box_h};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
               box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// As make_bf16_map_plain for bf16 or fp32 elements and rows `pitch` elements apart (pitch x
// element size a multiple of 16 bytes, pitch >= width).
inline bool make_map_pitched(CUtensorMap* map, const void* base, bool f32, uint64_t width,
                             uint64_t rows, uint64_t pitch, uint32_t box_w, uint32_t box_h) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {width, rows};
    const cuuint64_t strides[1] = {pitch * (f32 ? 4 : 2)};
    const cuuint32_t box[2] = {box_w, box_h};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
               const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE,
               box_w * (f32 ? 4 : 2) >= 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace gdr
