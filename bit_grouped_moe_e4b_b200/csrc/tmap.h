// 2-D and 3-D TMA tensor maps for the kernels' bulk copies.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace e4b {

// cuTensorMapEncodeTiled, looked up once through the runtime's driver entry
// point (the library does not link libcuda).
inline bool encode_tiled(CUtensorMap* m, CUtensorMapDataType dtype, uint32_t rank, const void* base,
                         const cuuint64_t* gdim, const cuuint64_t* gstride, const cuuint32_t* box,
                         CUtensorMapSwizzle swizzle) {
  using Fn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                          const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                          CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static Fn fn = nullptr;
  if (!fn) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return false;
    fn = reinterpret_cast<Fn>(ptr);
  }
  const cuuint32_t estride[3] = {1, 1, 1};
  return fn(m, dtype, rank, const_cast<void*>(base), gdim, gstride, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool encode_2d(CUtensorMap* m, CUtensorMapDataType dtype, const void* base, uint64_t inner,
                      uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
                      CUtensorMapSwizzle swizzle) {
  const cuuint64_t gdim[2] = {inner, outer};
  const cuuint64_t gstride[1] = {row_bytes};
  const cuuint32_t box[2] = {box_inner, box_outer};
  return encode_tiled(m, dtype, 2, base, gdim, gstride, box, swizzle);
}

// `planes` dense matrices [outer, inner] after one another; a box lies in one plane.
inline bool encode_planes(CUtensorMap* m, CUtensorMapDataType dtype, const void* base, uint64_t inner,
                          uint64_t outer, uint64_t planes, uint32_t value_bytes, uint32_t box_inner,
                          uint32_t box_outer, CUtensorMapSwizzle swizzle) {
  const cuuint64_t gdim[3] = {inner, outer, planes};
  const cuuint64_t gstride[2] = {inner * value_bytes, inner * outer * value_bytes};
  const cuuint32_t box[3] = {box_inner, box_outer, 1};
  return encode_tiled(m, dtype, 3, base, gdim, gstride, box, swizzle);
}

}  // namespace e4b
