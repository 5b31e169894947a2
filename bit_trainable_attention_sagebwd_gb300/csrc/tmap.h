// Host-side TMA tensor-map encoding (cuTensorMapEncodeTiled reached through the
// runtime's driver entry point, so the library links no libcuda stub).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

namespace sage {

inline PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

// 3-D tiled map, dims and box innermost first, strides in bytes between rows and between planes.  Returns false on
// error.
inline bool encode_tmap_3d(CUtensorMap* map, const void* base, CUtensorMapDataType dtype, const cuuint64_t (&dims)[3],
                           const cuuint64_t (&strides)[2], const cuuint32_t (&box)[3], CUtensorMapSwizzle swizzle) {
  auto enc = tmap_encoder();
  if (!enc) return false;
  cuuint32_t estr[3] = {1, 1, 1};
  auto encode = [&]() {
    return enc(map, dtype, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  if (r == CUDA_ERROR_INVALID_CONTEXT || r == CUDA_ERROR_NOT_INITIALIZED) {
    // a host thread that has not used its device yet: the encoding, unlike a call of the CUDA runtime, does not make
    // the device's context current by itself (cudaSetDevice does)
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = encode();
  }
  return r == CUDA_SUCCESS;
}

// 3-D tiled map over a contiguous [outer][rows][inner] tensor of `esize`-byte
// elements, box = [1][box_rows][box_inner].  With the default 128-byte swizzle
// box_inner * esize must be 128; without swizzle the box is a dense row-major
// [box_rows][box_inner] block in shared memory.  Out-of-range rows read as zero.
// Returns false on error.
inline bool make_tmap_3d(CUtensorMap* map, const void* base, CUtensorMapDataType dtype, int esize,
                         uint64_t inner, uint64_t rows, uint64_t outer, uint32_t box_inner,
                         uint32_t box_rows, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  return encode_tmap_3d(map, base, dtype, {inner, rows, outer},
                        {inner * (uint64_t)esize, inner * rows * (uint64_t)esize}, {box_inner, box_rows, 1}, swizzle);
}

}  // namespace sage
