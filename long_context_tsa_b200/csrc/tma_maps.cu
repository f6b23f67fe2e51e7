// TMA tensor-map encoding through the driver entry point (no link-time
// dependency on libcuda).
#include <cuda_runtime.h>

#include "tma_maps.h"

namespace tsa {
namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
  static EncodeTiled fn = nullptr;
  if (fn == nullptr) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiled>(ptr);
  }
  return fn;
}

bool encode(CUtensorMap* m, const void* base, uint64_t rows, int D, uint32_t box_rows,
            CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, int elem = 2) {
  EncodeTiled enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)D * elem};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / elem), box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(m, type, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool make_row_map(CUtensorMap* m, const void* base, uint64_t rows, int D) { return encode(m, base, rows, D, 1); }

bool make_tile_map(CUtensorMap* m, const void* base, uint64_t rows, int D, int box_rows) {
  return encode(m, base, rows, D, (uint32_t)box_rows);
}

bool make_code_map(CUtensorMap* m, const void* base, uint64_t rows, int box_rows) {
  return encode(m, base, rows, 128, (uint32_t)box_rows, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1);
}

}  // namespace tsa
