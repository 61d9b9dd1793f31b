// The distillation loss and its gradient (one translation unit per operator).
#include "launch_impl.cuh"

namespace specv {

cudaError_t launch_distill(int dtype, size_t smem, cudaStream_t s, const DistillParams& p) {
  return dtype == SPECV_BF16 ? launch_rows<distill_kernel<0>>(p.sp.C, p.N, smem, s, p)
                             : launch_rows<distill_kernel<1>>(p.sp.C, p.N, smem, s, p);
}

cudaError_t launch_distill_backward(int dtype, cudaStream_t s, const DistillParams& p) {
  const int vw = dtype == SPECV_BF16 ? Elem<0>::VW : Elem<1>::VW;
  const int chunks = (p.sp.V + vw - 2) / back_piece(vw) + 1;  // of a row that starts inside a vector
  const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(p.N) * chunks);
  const size_t smem = static_cast<size_t>(p.K) * 12;
  if (dtype == SPECV_BF16)
    distill_backward_kernel<0><<<blocks, kRowThreads, smem, s>>>(p, chunks);
  else
    distill_backward_kernel<1><<<blocks, kRowThreads, smem, s>>>(p, chunks);
  return cudaGetLastError();
}

}  // namespace specv
