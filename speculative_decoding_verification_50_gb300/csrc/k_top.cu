// The k largest logits (one translation unit per operator).
#include "launch_impl.cuh"

namespace specv {

cudaError_t launch_top_logits(int dtype, size_t smem, cudaStream_t s, const TopParams& p) {
  return dtype == SPECV_BF16 ? launch_rows<top_logits_kernel<0>>(p.sp.C, p.rows, smem, s, p)
                             : launch_rows<top_logits_kernel<1>>(p.sp.C, p.rows, smem, s, p);
}

}  // namespace specv
