// Launches of the product kernels.
#pragma once

#include <algorithm>
#include <atomic>
#include <mutex>

#include "api.cuh"
#include "product_kernel.cuh"

namespace specv {

// The largest size of a matrix that the kernels' 32-bit counts, rounded up to tiles or a CTA's
// threads, hold.
constexpr int32_t kProdMost = 0x7fffffff - 2047;

// A TMA descriptor of a matrix [batch][rows][cols] of 16-bit (or fp32) elements: boxes of
// `width` bytes x box_rows, swizzled over that width (128, 64; 0: 64 bytes, as they are),
// zeros outside.  base and the strides (bytes) are multiples of 16.
specv_status product_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t cols, int64_t rows,
                         int64_t batch, int64_t row_bytes, int64_t batch_bytes, int box_rows, int width = 128);

// An operand: K-major [rows of A or B][K], or MN-major [K][rows of A or B].
inline specv_status operand_map(CUtensorMap* map, bool bf16, bool mn, const void* base, int64_t cols, int64_t rows,
                                int64_t batch, int64_t stride, int64_t batch_stride, int box_rows = 0) {
  return product_map(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, base, cols, rows, batch,
                     2 * stride, 2 * batch_stride, box_rows ? box_rows : mn ? kProdBK : kProdHalf);
}

// A launch that may be scheduled while the one before it on the stream drains (it waits
// for it with griddepcontrol.wait).
template <typename Kern, typename Params>
cudaError_t launch_grid(Kern k, dim3 blocks, int threads, cudaStream_t stream, const Params& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = blocks;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, p);
}

// Tiles of a product: of 256 x 256, or of half of that.
inline int64_t product_units(const ProductParams& p, int tile) {
  const int64_t tm = (static_cast<int64_t>(p.M) + tile - 1) / tile, tn = (static_cast<int64_t>(p.N) + tile - 1) / tile;
  return (p.symmetric ? tm * (tm + 1) / 2 : tm * tn) * p.batch * p.splits;
}

// CTAs of a product: as many as the GPU holds, or as there are units of work.
template <bool PAIR>
int product_grid(const ProductParams& p) {
  constexpr int ctas = PAIR ? 2 : 1;
  return static_cast<int>(ctas * std::min<int64_t>(product_units(p, PAIR ? kProdTile : kProdHalf), api_sm_count() / ctas));
}

template <bool PAIR, bool A_MN, bool B_MN, class Epi>
cudaError_t launch_product(ProductParams& p, const typename Epi::Params& e, cudaStream_t stream) {
  constexpr int kDevices = 64;
  constexpr int smem = kProdSmem<Epi::kStaging>;
  static std::atomic<bool> allowed[kDevices];
  auto kern = product_kernel<PAIR, A_MN, B_MN, Epi>;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= kDevices || !allowed[dev].load(std::memory_order_acquire)) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    if (dev < kDevices) allowed[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(product_grid<PAIR>(p)), 1, 1);
  cfg.blockDim = dim3(kProdThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = PAIR ? 2 : 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  p.tn = (p.N + (PAIR ? kProdTile : kProdHalf) - 1) / (PAIR ? kProdTile : kProdHalf);
  p.idesc = prod_idesc(p.bf16, A_MN, B_MN, PAIR ? kProdTile : kProdHalf);
  return cudaLaunchKernelEx(&cfg, kern, p, e);
}

}  // namespace specv
