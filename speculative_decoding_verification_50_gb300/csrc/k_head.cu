// The kernels of the head's loss: products with their epilogues, and the rows around them.
#include "head_kernel.cuh"
#include "head_launch.cuh"
#include "product_launch.cuh"

namespace specv {

namespace {

// Row r's target if it counts, else -1.
__device__ __forceinline__ int head_target(const HeadRowsParams& p, int r) {
  const int t = p.target[r];
  if (t < 0 || t >= p.V || (p.weight && p.weight[r] == 0.f)) return -1;
  if (p.stats) {
    const float lse = p.stats[2LL * r], nll = p.stats[2LL * r + 1];
    if (!(lse - lse == 0.f) || !(nll - nll == 0.f)) return -1;
  }
  return t;
}
// Its gradient's weight.
__device__ __forceinline__ float head_weight(const HeadRowsParams& p, int r) {
  return (p.weight ? p.weight[r] : 1.f) * (p.up ? p.up[r] : 1.f) * p.scale;
}
// Whether a row's log-sum-exp does not hold its probabilities' digits.
__device__ __forceinline__ bool head_far(float lse) { return fabsf(lse) * kLog2e > kFarRow; }
__device__ __forceinline__ HeadRow head_row(float lse, float nll, float g, int target) {
  return {0.f, lse * kLog2e, g, g * expm1f(-nll), target, head_far(lse) ? 0.f : pos_inf(), {0, 0}};
}
// The largest weight of a CTA's threads (a power of two of them up to 1024).
__device__ __forceinline__ float head_most(float g, float (&warps)[32]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = g;
  __syncthreads();
  for (int k = 0; k < static_cast<int>(blockDim.x) / 32; ++k) g = fmaxf(g, warps[k]);
  return g > 0.f && g < pos_inf() ? g : 1.f;
}

}  // namespace

// Which rows count, and where they go (in order).  One CTA.
__global__ void __launch_bounds__(kRowsThreads, 1) head_rows_kernel(const HeadRowsParams p) {
  __shared__ int warps[32];
  __shared__ float weights[32];
  __shared__ int before;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) before = 0;
  pdl_wait_primary();
  pdl_launch_dependents();
  float most = 0.f;
  for (int r = threadIdx.x; r < p.N; r += kRowsThreads)
    if (head_target(p, r) >= 0) most = fmaxf(most, fabsf(head_weight(p, r)));
  most = head_most(most, weights);
  if (threadIdx.x == 0) *p.most = most;
  for (int first = 0; first < p.N; first += kRowsThreads) {
    const int r = first + threadIdx.x;
    const int target = r < p.N ? head_target(p, r) : -1;
    const bool use = target >= 0 || (p.all && r < p.N && p.target[r] == -1 && !(p.weight && p.weight[r] == 0.f));
    const unsigned votes = __ballot_sync(0xffffffffu, use);
    if (lane == 0) warps[warp] = __popc(votes);
    __syncthreads();
    if (warp == 0) {
      const int n = warps[lane];
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      warps[lane] = before + x - n;
      __syncwarp();
      if (lane == 31) before += x;
    }
    __syncthreads();
    const int at = use ? warps[warp] + __popc(votes & ((1u << lane) - 1)) : -1;
    __syncthreads();
    if (r < p.N) {
      p.place[r] = at;
      if (at >= 0) {
        p.source[at] = r;
        p.use_target[at] = target;
        if (p.row) p.row[at] = head_row(p.stats[2LL * r], p.stats[2LL * r + 1], head_weight(p, r) / most, target);
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) *p.count = before;
}

// A row of 16-bit values per CTA: the rows in use brought together at 16-byte boundaries.
// Bound by bytes (2 x 2 D per row).
__global__ void __launch_bounds__(kGatherThreads) head_gather_kernel(const HeadGatherParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  __shared__ float weights[32];
  const int n = p.count ? *p.count : p.N;
  if (p.late && blockIdx.x == 0 && threadIdx.x == 0) *p.late = 0;
  float most = 1.f;
  if (p.info.most) {  // (up to 256 rows, which every CTA looks through)
    const int r = threadIdx.x;
    most = head_most(r < n && head_target(p.info, r) >= 0 ? fabsf(head_weight(p.info, r)) : 0.f, weights);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.info.most = most;
  }
  const int all = (n + p.pad_to - 1) / p.pad_to * p.pad_to;
  for (int i = blockIdx.x; i < max(all, p.pad_to); i += gridDim.x) {
    if (p.info.row && threadIdx.x == 0 && i < n) {
      const int t = head_target(p.info, i);
      p.info.row[i] = t < 0 ? head_no_row()
                            : head_row(p.info.stats[2LL * i], p.info.stats[2LL * i + 1], head_weight(p.info, i) / most, t);
    }
    uint16_t* out = p.out + i * p.out_stride;
    const int D8 = (p.D + 7) / 8;
    const uint16_t* in = i < n ? p.in + static_cast<int64_t>(p.source ? p.source[i] : i) * p.in_stride : nullptr;
    auto get = [&](int j) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (!in) return v;
      if (p.vec && 8 * j + 8 <= p.D) return __ldg(reinterpret_cast<const uint4*>(in) + j);
      uint32_t h[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) h[k] = 8 * j + k < p.D ? in[8 * j + k] : 0u;
      return make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    };
    bool bad = false;
    if (p.bad && in) {
      for (int j = threadIdx.x; j < D8; j += kGatherThreads) {
        const uint4 v = get(j);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) bad |= (w[k] & 0x7f80u) == 0x7f80u || (w[k] & 0x7f800000u) == 0x7f800000u;
      }
    }
    bad = __syncthreads_or(bad);
    if (p.bad && in && threadIdx.x == 0) p.bad[i] = bad;
    for (int j = threadIdx.x; j < D8; j += kGatherThreads)
      reinterpret_cast<uint4*>(out)[j] = bad ? make_uint4(0, 0, 0, 0) : get(j);
    if (p.stats && in) {
      // A row far from zero: nll, where that is smaller than |lse|, and the target's logit.
      const int r = p.source ? p.source[i] : i, t = p.source ? p.target[i] : head_target(p.info, i);
      const float lse = p.stats[2LL * r], nll = p.stats[2LL * r + 1];
      if (t >= 0 && head_far(lse) && nll < fabsf(lse)) {  // (the CTA's)
        float sum = 0.f;
        const uint16_t* w = p.head + t * p.head_stride;
        for (int j = threadIdx.x; j < p.D; j += kGatherThreads)
          sum = fmaf(__uint_as_float(static_cast<uint32_t>(in[j]) << 16), __uint_as_float(static_cast<uint32_t>(w[j]) << 16), sum);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) weights[threadIdx.x >> 5] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
#pragma unroll
          for (int k = 1; k < kGatherThreads / 32; ++k) sum += weights[k];
          p.row[i].ref = sum;
          p.row[i].off = nll * kLog2e;
        }
      }
    }
  }
}

// RB rows per CTA, 256 / RB threads each: the parts of a row joined, its loss and what the
// backward pass reads.
template <int RB>
__global__ void __launch_bounds__(kJoinThreads) head_join_kernel(const HeadJoinParams p) {
  constexpr int T = kJoinThreads / RB;
  __shared__ float2 got[kJoinThreads];
  __shared__ int failed;
  if (threadIdx.x == 0) failed = 0;
  pdl_wait_primary();
  pdl_launch_dependents();
  __syncthreads();
  for (int i = threadIdx.x; i < p.errs; i += kJoinThreads)
    if (p.err[i]) failed = 1;
  const int r = blockIdx.x * RB + threadIdx.x % RB, k = threadIdx.x / RB;
  const int t = r < p.N ? p.target[r] : -1;
  const float w = r < p.N && p.weight ? p.weight[r] : 1.f;
  const bool use = (t >= 0 || (p.all && t == -1 && r < p.N)) && t < p.V && w != 0.f;
  const int at = r < p.N ? (p.place ? p.place[r] : r) : -1;
  const float c2 = p.scale * kLog2e;
  float m = kNegMax, s = 0.f;
  if (use && at >= 0) {
    for (int j = k; j < p.parts; j += 8 * T) {
      float2 x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) x[u] = j + u * T < p.parts ? p.part[(j + u * T) * p.ld + at] : make_float2(kNegMax, 0.f);
#pragma unroll
      for (int u = 0; u < 8; ++u) soft_join(m, s, x[u].x, x[u].y, c2);
    }
  }
  if (RB == 1) {  // a row's threads: within warps, then over the warps
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      soft_join(m, s, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o), c2);
    if ((threadIdx.x & 31) == 0) got[threadIdx.x >> 5] = make_float2(m, s);
    __syncthreads();
    if (threadIdx.x == 0)
#pragma unroll
      for (int o = 1; o < kJoinThreads / 32; ++o) soft_join(m, s, got[o].x, got[o].y, c2);
  } else {
    got[threadIdx.x] = make_float2(m, s);
    __syncthreads();
#pragma unroll
    for (int o = T / 2; o > 0; o >>= 1) {
      if (k < o) {
        const float2 x = got[threadIdx.x + o * RB];
        soft_join(m, s, x.x, x.y, c2);
        got[threadIdx.x] = make_float2(m, s);
      }
      __syncthreads();
    }
  }
  if (k != 0 || r >= p.N) return;
  float lse = 0.f, nll = 0.f, loss = 0.f;
  int status = (t < -1 || t >= p.V) && w != 0.f ? kBadToken : 0;
  HeadRow row = head_no_row();
  if (use && t < 0) {
    lse = s == 0.f ? neg_inf() : p.scale * m + logf(s);
    if (failed) status |= kTimeout;
  } else if (use) {
    const float zt = p.z_target[at], d2 = (m - zt) * c2;
    // (relative to the target's logit where that is the largest, else to the largest of the others)
    nll = s == 0.f ? 0.f : d2 <= 0.f ? log1pf(s * exp2f(d2)) : d2 * kLn2 + logf(s + exp2f(-d2));
    if (d2 == pos_inf()) nll = (m - zt) * p.scale;  // (a difference up to fp32's range, but not times log2(e))
    lse = p.scale * zt + nll;
    if (failed) status |= kTimeout;
    if (p.bad && p.bad[at]) status |= kNonFinite;
    if (!(s - s == 0.f) || !(lse - lse == 0.f)) status |= kNonFinite;
    if (!status) {
      loss = w * nll;
      if (p.row) row = head_row(lse, nll, w * p.scale / *p.most, t);
      if (p.row && head_far(lse)) {  // relative to the largest logit
        row.ref = s == 0.f || d2 <= 0.f ? zt : m;
        row.off = s == 0.f || d2 <= 0.f ? nll * kLog2e : log2f(s + exp2f(-d2));
      }
    }
  }
  if (status) lse = nll = __int_as_float(0x7fc00000);
  p.loss[r] = loss;
  if (p.stats) {
    p.stats[2LL * r] = lse;
    p.stats[2LL * r + 1] = nll;
  }
  if (p.status) p.status[r] = status;
  if (p.row && at >= 0) p.row[at] = row;
}

// dz from the weights that were kept, in their place (fp16 in, bf16 out).  A warp takes 256
// columns of a row.  Bound by bytes (4 per logit).
__global__ void __launch_bounds__(256) head_weight_kernel(const HeadWeightParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int n = p.count ? *p.count : p.N, rows = max((n + kProdBK - 1) / kProdBK * kProdBK, kProdBK);
  const int lane = threadIdx.x & 31, pieces = (p.V + 255) / 256;
  const int64_t all = static_cast<int64_t>(rows) * pieces;
  for (int64_t x = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); x < all; x += static_cast<int64_t>(gridDim.x) * 8) {
    const int i = static_cast<int>(x / pieces), col = static_cast<int>(x - static_cast<int64_t>(i) * pieces) * 256 + lane * 8;
    if (col >= p.V) continue;
    uint4* at = reinterpret_cast<uint4*>(p.w + i * p.stride + col);
    uint4 v = make_uint4(0, 0, 0, 0);
    const HeadRow r = i < n ? p.row[i] : head_no_row();
    if (r.g != 0.f) {
      v = __ldcs(at);
      const float f = r.g * ex2(fmaf(p.part[(col / p.part_cols) * p.ld + i].x - r.ref, p.c2, -r.off));
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        // (the weights' scale is taken off them, not off f: that would be 0 from 2^-111 on, in the
        // place of 2^-126)
        float a = e.x * kUnkeep * f, b = e.y * kUnkeep * f;
        if (col + 2 * k == r.target) a = r.at;
        if (col + 2 * k + 1 == r.target) b = r.at;
        w[k] = pack_bf16(a, b);
      }
      v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    *at = v;
  }
}

// dh from the sums of K's parts, rows back in their places; nothing but zeros after a late product.
__global__ void __launch_bounds__(256) head_finish_kernel(const HeadFinishParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const bool late = *p.late != 0;
  if (late) {
    const int64_t first = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, step = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t r = first; p.status && r < p.N; r += step) p.status[r] |= kTimeout;
    for (int64_t x = first; p.head && x < static_cast<int64_t>(p.V) * p.D; x += step) {
      const int64_t v = x / p.D;
      p.head[v * p.head_stride + (x - v * p.D)] = 0;
    }
  }
  if (!p.out) return;
  const int D4 = (p.D + 3) / 4;
  const float f = *p.most;
  const int64_t all = static_cast<int64_t>(p.N) * D4;
  for (int64_t x = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; x < all; x += static_cast<int64_t>(gridDim.x) * 256) {
    const int r = static_cast<int>(x / D4), j = static_cast<int>(x - static_cast<int64_t>(r) * D4) * 4;
    const int at = p.place ? p.place[r] : r;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (at >= 0 && p.row[at].g != 0.f && !late) {
#pragma unroll 16
      for (int k = 0; k < p.splits; ++k) {
        const float4 a = __ldcs(reinterpret_cast<const float4*>(p.sum + k * p.split_stride + at * p.ld + j));
        v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
      }
    }
    uint16_t* out = p.out + r * p.stride + j;
    const uint2 w = make_uint2(pack_bf16(v.x * f, v.y * f), pack_bf16(v.z * f, v.w * f));
    if (p.vec && j + 4 <= p.D) {
      *reinterpret_cast<uint2*>(out) = w;
    } else {
      const uint32_t h[2] = {w.x, w.y};
      for (int k = 0; k < min(4, p.D - j); ++k) out[k] = static_cast<uint16_t>(h[k / 2] >> (16 * (k & 1)));
    }
  }
}

// Up to 128 rows: tiles of 128 x 128.
static bool few(const ProductParams& p) { return p.M <= kProdHalf; }
static int stats_chunk(const ProductParams& p) { return p.M <= kProdTile ? kStatsChunkFew : kStatsChunk; }

template <bool LONG>
static cudaError_t launch_stats_of(ProductParams& p, const HeadStatsParams& e, cudaStream_t s) {
  return few(p) ? launch_product<false, false, false, StatsEpi<LONG, kProdHalf / 2>>(p, e, s)
                : launch_product<true, false, false, StatsEpi<LONG, kProdTile / 2>>(p, e, s);
}
cudaError_t launch_head_stats(ProductParams& p, const HeadStatsParams& e, cudaStream_t s) {
  p.chunk = stats_chunk(p);
  return p.K <= p.chunk * kProdBK ? launch_stats_of<false>(p, e, s) : launch_stats_of<true>(p, e, s);
}
cudaError_t launch_head_keep(ProductParams& p, const HeadStatsParams& e, const Out16& out, cudaStream_t s) {
  p.chunk = stats_chunk(p);
  return few(p) ? launch_product<false, false, false, KeepEpi<kProdHalf / 2>>(p, {e, out}, s)
                : launch_product<true, false, false, KeepEpi<kProdTile / 2>>(p, {e, out}, s);
}
cudaError_t launch_head_weight(const HeadWeightParams& p, int blocks, cudaStream_t s) {
  return launch_grid(head_weight_kernel, blocks, 256, s, p);
}
cudaError_t launch_head_prob(ProductParams& p, const ProbEpi::Params& e, cudaStream_t s) {
  return few(p) ? launch_product<false, false, false, ProbEpi>(p, e, s) : launch_product<true, false, false, ProbEpi>(p, e, s);
}
cudaError_t launch_head_hidden(ProductParams& p, const SumEpi::Params& e, cudaStream_t s) {
  return few(p) ? launch_product<false, false, true, SumEpi>(p, e, s) : launch_product<true, false, true, SumEpi>(p, e, s);
}
cudaError_t launch_head_head(ProductParams& p, const Out16& out, const float* factor, cudaStream_t s) {
  if (p.K <= 16 * kProdBK) return launch_product<true, true, true, StoreEpi<true>>(p, {out, factor}, s);
  return launch_product<true, true, true, StoreEpi<false>>(p, {out, factor}, s);
}
cudaError_t launch_head_rows(const HeadRowsParams& p, cudaStream_t s) {
  return launch_grid(head_rows_kernel, 1, kRowsThreads, s, p);
}
cudaError_t launch_head_gather(const HeadGatherParams& p, int blocks, cudaStream_t s) {
  return launch_grid(head_gather_kernel, blocks, kGatherThreads, s, p);
}
cudaError_t launch_head_join(const HeadJoinParams& p, cudaStream_t s) {
  return p.N <= 1024 ? launch_grid(head_join_kernel<1>, p.N, kJoinThreads, s, p)
                     : launch_grid(head_join_kernel<32>, (p.N + 31) / 32, kJoinThreads, s, p);
}
cudaError_t launch_head_finish(const HeadFinishParams& p, int blocks, cudaStream_t s) {
  return launch_grid(head_finish_kernel, blocks, 256, s, p);
}

}  // namespace specv
