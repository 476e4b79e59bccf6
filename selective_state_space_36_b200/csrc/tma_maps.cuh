// tma_maps.cuh -- host side of the tiled TMA copies: tensor maps of (batch,
// seqlen, width) bf16 tensors.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace ssm {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                                   CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                   CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled, fetched through the runtime (no link-time
// dependency on the driver library); null if the driver has none.
inline EncodeTiledFn encode_tiled_fn() {
    static EncodeTiledFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            return (EncodeTiledFn) nullptr;
        }
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}

// A dense bf16 tensor of D dimensions, innermost first, as a tiled map with boxes
// of `boxes` elements; what lies outside the tensor reads as zeros and is not
// written by stores.
template <int D>
bool encode_bf16(CUtensorMap *m, const void *p, const int64_t (&n)[D], const int (&boxes)[D], CUtensorMapSwizzle sw) {
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return false;
    cuuint64_t dims[D], strides[D - 1], bytes = 2;
    cuuint32_t box[D], es[D];
    for (int i = 0; i < D; ++i) {
        dims[i] = (cuuint64_t)n[i];
        box[i] = (cuuint32_t)boxes[i];
        es[i] = 1;
        bytes *= dims[i];
        if (i < D - 1) strides[i] = bytes;
    }
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, D, const_cast<void *>(p), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A (batch, seqlen, width) bf16 tensor as a 3-D tiled map: boxes of 64
// elements of the width x `steps` steps x 1 row, 128-byte swizzle; steps past
// the sequence read as zeros and are not written by stores.
inline bool encode_btw(CUtensorMap *m, const void *p, int64_t batch, int64_t seqlen, int64_t width, int steps) {
    return encode_bf16<3>(m, p, {width, seqlen, batch}, {64, steps, 1}, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace ssm
