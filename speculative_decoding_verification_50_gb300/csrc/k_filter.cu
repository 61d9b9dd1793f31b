// Filtered sampling: one translation unit per operator, compiled in parallel.
#include "launch_impl.cuh"

namespace specv {

cudaError_t launch_sample_filter(int dtype, size_t smem, cudaStream_t s, const FilterParams& p) {
  return dtype == SPECV_BF16 ? launch_rows<sample_filter_kernel<0>>(p.sp.C, p.rows, smem, s, p)
                             : launch_rows<sample_filter_kernel<1>>(p.sp.C, p.rows, smem, s, p);
}

}  // namespace specv
