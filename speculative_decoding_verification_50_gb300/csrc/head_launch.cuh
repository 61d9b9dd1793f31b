// Launchers of the head's loss (k_head.cu), and TMA descriptors for the products.
#pragma once

#include "head_kernel.cuh"

namespace specv {

// in chunks of kStatsChunk blocks where D is longer
cudaError_t launch_head_stats(ProductParams& p, const HeadStatsParams& e, cudaStream_t s);
cudaError_t launch_head_keep(ProductParams& p, const HeadStatsParams& e, const Out16& out, cudaStream_t s);
cudaError_t launch_head_weight(const HeadWeightParams& p, int blocks, cudaStream_t s);
cudaError_t launch_head_prob(ProductParams& p, const ProbEpi::Params& e, cudaStream_t s);
cudaError_t launch_head_hidden(ProductParams& p, const SumEpi::Params& e, cudaStream_t s);
cudaError_t launch_head_head(ProductParams& p, const Out16& out, const float* factor, cudaStream_t s);
cudaError_t launch_head_rows(const HeadRowsParams& p, cudaStream_t s);
cudaError_t launch_head_gather(const HeadGatherParams& p, int blocks, cudaStream_t s);
cudaError_t launch_head_join(const HeadJoinParams& p, cudaStream_t s);
cudaError_t launch_head_finish(const HeadFinishParams& p, int blocks, cudaStream_t s);

}  // namespace specv
