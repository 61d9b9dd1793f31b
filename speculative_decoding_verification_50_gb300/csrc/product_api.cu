// TMA descriptors of the product kernels' operands.
#include <cudaTypedefs.h>

#include "product_launch.cuh"

namespace specv {

specv_status product_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t cols, int64_t rows,
                         int64_t batch, int64_t row_bytes, int64_t batch_bytes, int box_rows, int width) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  if (!encode) return api_fail(SPECV_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const int es = type == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(batch)};
  if (batch == 1) batch_bytes = (row_bytes * rows + 15) / 16 * 16;
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(batch_bytes)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>((width ? width : 64) / es), static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t step[3] = {1, 1, 1};
  const CUresult r = encode(map, type, 3, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            width == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                            : width == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                          : CU_TENSOR_MAP_SWIZZLE_NONE,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return api_fail(SPECV_ERR_CUDA, "cuTensorMapEncodeTiled: error %d", static_cast<int>(r));
  return SPECV_OK;
}

}  // namespace specv
