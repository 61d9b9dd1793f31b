// Launches of the product kernels.
#pragma once

#include <atomic>
#include <mutex>

#include "api.cuh"
#include "product_kernel.cuh"

namespace specv {

// A TMA descriptor of a matrix [batch][rows][cols] of 16-bit (or fp32) elements: boxes of
// box_cols (128 bytes) x box_rows under the 128-byte swizzle, zeros outside.  base and the
// strides (bytes) are multiples of 16.
specv_status product_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t cols, int64_t rows,
                         int64_t batch, int64_t row_bytes, int64_t batch_bytes, int box_rows);

// An operand: K-major [rows of A or B][K], or MN-major [K][rows of A or B].
inline specv_status operand_map(CUtensorMap* map, bool bf16, bool mn, const void* base, int64_t cols, int64_t rows,
                                int64_t batch, int64_t stride, int64_t batch_stride) {
  return product_map(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, base, cols, rows, batch,
                     2 * stride, 2 * batch_stride, mn ? kProdBK : kProdHalf);
}

// A launch that may be scheduled while the one before it on the stream drains (it waits
// for it with griddepcontrol.wait).
template <typename Kern, typename Params>
cudaError_t launch_grid(Kern k, int blocks, int threads, cudaStream_t stream, const Params& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, p);
}

// CTAs of a product: as many pairs as the GPU holds, or one pair per unit of work where
// those are fewer.
inline int product_grid(const ProductParams& p) {
  const int64_t tm = (static_cast<int64_t>(p.M) + kProdTile - 1) / kProdTile;
  const int64_t units = (p.symmetric ? tm * (tm + 1) / 2 : tm * p.tn) * p.batch * p.splits;
  const int64_t pairs = api_sm_count() / 2;
  return static_cast<int>(2 * (units < pairs ? units : pairs));
}

template <bool A_MN, bool B_MN, class Epi>
cudaError_t launch_product(ProductParams& p, const typename Epi::Params& e, cudaStream_t stream) {
  constexpr int kDevices = 64;
  constexpr int smem = kProdSmem<Epi::kStaging>;
  static std::atomic<bool> allowed[kDevices];
  auto kern = product_kernel<A_MN, B_MN, Epi>;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= kDevices || !allowed[dev].load(std::memory_order_acquire)) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    if (dev < kDevices) allowed[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(product_grid(p)), 1, 1);
  cfg.blockDim = dim3(kProdThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];  // (the kernel is compiled for clusters of two)
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p, e);
}

}  // namespace specv
