// Launchers of the orthogonalised update (k_orth.cu).
#pragma once

#include "orth_kernel.cuh"
#include "orth_small.cuh"

namespace specv {

// B clusters of C CTAs
cudaError_t launch_orth_small(int dtype, const SmallParams& p, int C, int B, cudaStream_t s);
cudaError_t launch_orth_squares(int dtype, const OrthInParams& p, cudaStream_t s);
cudaError_t launch_orth_scale(int dtype, const OrthInParams& p, cudaStream_t s);
// mn: the operands as they lie are [K][rows]; half: tiles of 128 x 128
template <bool FINE>
cudaError_t launch_orth_gram(bool half, bool mn, ProductParams& p, const typename SymEpi<false, FINE>::Params& e, cudaStream_t s);
cudaError_t launch_orth_sums(bool half, bool mn, ProductParams& p, const SumEpi::Params& e, cudaStream_t s);
cudaError_t launch_orth_join(const OrthJoinParams& p, int B, cudaStream_t s);
template <bool FINE>
cudaError_t launch_orth_poly(bool half, ProductParams& p, const typename SymEpi<true, FINE>::Params& e, cudaStream_t s);
cudaError_t launch_orth_step(bool half, bool mn, ProductParams& p, const StepEpi<false>::Params& e, cudaStream_t s);
cudaError_t launch_orth_last(bool half, bool mn, ProductParams& p, const StepEpi<true>::Params& e, cudaStream_t s);

}  // namespace specv
