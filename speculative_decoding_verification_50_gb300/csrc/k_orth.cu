// The kernels of the orthogonalised update.
#include "orth_launch.cuh"
#include "orth_squares.cuh"
#include "product_launch.cuh"

namespace specv {

namespace {

// Vector j of a row: VW elements, zeros past its end.
template <int DT>
__device__ __forceinline__ typename Elem<DT>::Vec row_vec(const void* row, int64_t j, int64_t cols, bool vec) {
  constexpr int VW = Elem<DT>::VW;
  if (vec && (j + 1) * VW <= cols) return Elem<DT>::vec(row, j * VW);
  union {
    typename Elem<DT>::Raw e[VW];
    typename Elem<DT>::Vec v;
  } x;
#pragma unroll
  for (int k = 0; k < VW; ++k) x.e[k] = j * VW + k < cols ? Elem<DT>::raw(row, j * VW + k) : typename Elem<DT>::Raw(0);
  return x.v;
}

// use(row, vector, load(row, vector)) over this CTA's share of a matrix's rows of nv vectors:
// a share of a long row's vectors per CTA (rows without gaps are one), or rows in turn.  Four
// loads are under way before the first is used.
template <typename V, typename L, typename U>
__device__ __forceinline__ void each_vec(const OrthInParams& p, int64_t nv, L&& load, U&& use) {
  constexpr int kAhead = 4;
  int64_t r = 0, rows = 1, row_step = 1, j0 = static_cast<int64_t>(blockIdx.x) * kOrthThreads + threadIdx.x,
          step = static_cast<int64_t>(gridDim.x) * kOrthThreads;
  if (p.rows > 1) {
    // a row per `step` threads, the power of two that is at most its vectors
    int lanes = 32;
    while (lanes < kOrthThreads && 2 * lanes <= nv) lanes *= 2;
    const int per = kOrthThreads / lanes;
    r = static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / lanes, rows = p.rows;
    row_step = static_cast<int64_t>(gridDim.x) * per, j0 = threadIdx.x % lanes, step = lanes;
  }
  for (; r < rows; r += row_step)
    for (int64_t j = j0; j < nv; j += kAhead * step) {
      V x[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (j + u * step < nv) x[u] = load(r, j + u * step);
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (j + u * step < nv) use(r, j + u * step, x[u]);
    }
}

template <int DT>
__device__ __forceinline__ const void* row_at(const OrthInParams& p, int z, int64_t r) {
  return static_cast<const char*>(p.in) + (z * p.batch_stride + r * p.row_stride) * Elem<DT>::ES;
}

}  // namespace

// Sums of squares of a matrix's parts, at the scale of their largest entries (neither tiny
// nor huge entries leave fp32's range).  Bound by bytes.
template <int DT>
__global__ void __launch_bounds__(kOrthThreads) orth_squares_kernel(const OrthInParams p) {
  __shared__ ScaledSquares warps[kOrthThreads / 32], sum;
  pdl_wait_primary();
  pdl_launch_dependents();
  constexpr int VW = Elem<DT>::VW;
  const int z = blockIdx.y;
  const int64_t nv = (p.cols + VW - 1) / VW;
  ScaledSquares a = {kSquaresLeast, 0.f};
  float inv = 1.f / kSquaresLeast;
  using Vec = typename Elem<DT>::Vec;
  each_vec<Vec>(
      p, nv, [&](int64_t r, int64_t j) { return row_vec<DT>(row_at<DT>(p, z, r), j, p.cols, p.vec); },
      [&](int64_t, int64_t, const Vec& w) {
        float x[VW];
        Elem<DT>::unpack(w, x);
        squares_add<VW>(a, inv, x);
      });
  squares_cta(a, warps, sum);
  if (threadIdx.x == 0) p.part[z * p.blocks + blockIdx.x] = sum;
}

// X = G / |G| in fp16 and what that leaves out; zeros for a matrix that is zero, or not
// finite (flagged).
template <int DT>
__global__ void __launch_bounds__(kOrthThreads) orth_scale_kernel(const OrthInParams p) {
  __shared__ ScaledSquares warps[kOrthThreads / 32], sum;
  pdl_wait_primary();
  pdl_launch_dependents();
  constexpr int VW = Elem<DT>::VW;
  const int z = blockIdx.y;
  ScaledSquares a = {kSquaresLeast, 0.f};
  for (int k = threadIdx.x; k < p.blocks; k += kOrthThreads) squares_join(a, p.part[z * p.blocks + k]);
  squares_cta(a, warps, sum);
  const float root = sqrtf(sum.s);
  const bool bad = !(sum.s < pos_inf());
  const float inv = 1.f / sum.m, f = bad || sum.s == 0.f ? 0.f : p.scale / root;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (p.norm) p.norm[z] = bad ? __int_as_float(0x7fc00000) : sum.m * root;
    if (p.status) p.status[z] = bad ? kNonFinite : 0;
  }
  using Vec = typename Elem<DT>::Vec;
  auto load = [&](int64_t r, int64_t j) { return row_vec<DT>(row_at<DT>(p, z, r), j, p.cols, p.vec); };
  each_vec<Vec>(p, p.ld / VW, load, [&](int64_t r, int64_t j, const Vec& raw) {
    float x[VW];
    Elem<DT>::unpack(raw, x);
    uint32_t hi[VW / 2], lo[VW / 2];
#pragma unroll
    for (int k = 0; k < VW / 2; ++k) {
      const float u = bad ? 0.f : x[2 * k] * inv * f, v = bad ? 0.f : x[2 * k + 1] * inv * f;
      hi[k] = pack_f16(u, v);
      const float2 g = unpack_f16(hi[k]);
      lo[k] = pack_f16(u - g.x, v - g.y);
    }
    const int64_t at = z * p.matrix + r * p.ld + j * VW;
    if constexpr (VW == 8) {
      *reinterpret_cast<uint4*>(p.hi + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(p.lo + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    } else {
      *reinterpret_cast<uint2*>(p.hi + at) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(p.lo + at) = make_uint2(lo[0], lo[1]);
    }
  });
}

__global__ void __launch_bounds__(256) orth_join_kernel(const OrthJoinParams p) {
  __shared__ uint16_t turned[2][64][72];
  pdl_wait_primary();
  pdl_launch_dependents();
  int u = blockIdx.x, pi = 0;
  for (; u >= p.patches - pi; ++pi) u -= p.patches - pi;
  const int pj = pi + u, z = blockIdx.y;
  const int64_t matrix = p.n * p.ld;
  const float* sum = p.sum + z * p.splits * matrix;
  const int c = (threadIdx.x & 15) * 4, j = pj * 64 + c;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = k * 16 + (threadIdx.x >> 4), i = pi * 64 + r;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < p.n && j < p.n) {  // (ld is a multiple of 8: words at the end of a row are whole)
#pragma unroll 4
      for (int q = 0; q < p.splits; ++q) {
        const float4 o = __ldcs(reinterpret_cast<const float4*>(sum + q * matrix + i * p.ld + j));
        x.x += o.x, x.y += o.y, x.z += o.z, x.w += o.w;
      }
    }
    x.x *= p.alpha, x.y *= p.alpha, x.z *= p.alpha, x.w *= p.alpha;
    const uint32_t h[2] = {pack_f16(x.x, x.y), pack_f16(x.z, x.w)};
    const float2 g0 = unpack_f16(h[0]), g1 = unpack_f16(h[1]);
    const uint32_t l[2] = {pack_f16(x.x - g0.x, x.y - g0.y), pack_f16(x.z - g1.x, x.w - g1.y)};
    if (i < p.n && j < p.n) {
      const int64_t at = z * matrix + i * p.ld + j;
      *reinterpret_cast<uint2*>(p.hi + at) = make_uint2(h[0], h[1]);
      if (p.lo) *reinterpret_cast<uint2*>(p.lo + at) = make_uint2(l[0], l[1]);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      turned[0][c + t][r] = static_cast<uint16_t>(h[t >> 1] >> (16 * (t & 1)));
      turned[1][c + t][r] = static_cast<uint16_t>(l[t >> 1] >> (16 * (t & 1)));
    }
  }
  if (pi == pj) return;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = k * 16 + (threadIdx.x >> 4), i = pj * 64 + r, jj = pi * 64 + c;
    if (i >= p.n) continue;
    const int64_t at = z * matrix + i * p.ld + jj;
    *reinterpret_cast<uint2*>(p.hi + at) = *reinterpret_cast<const uint2*>(&turned[0][r][c]);
    if (p.lo) *reinterpret_cast<uint2*>(p.lo + at) = *reinterpret_cast<const uint2*>(&turned[1][r][c]);
  }
}

template <typename Kern>
static cudaError_t launch_in(Kern k, const OrthInParams& p, cudaStream_t s) {
  return launch_grid(k, dim3(p.blocks, p.batch, 1), kOrthThreads, s, p);
}

cudaError_t launch_orth_squares(int dtype, const OrthInParams& p, cudaStream_t s) {
  return dtype == SPECV_BF16 ? launch_in(orth_squares_kernel<0>, p, s) : launch_in(orth_squares_kernel<1>, p, s);
}
cudaError_t launch_orth_scale(int dtype, const OrthInParams& p, cudaStream_t s) {
  return dtype == SPECV_BF16 ? launch_in(orth_scale_kernel<0>, p, s) : launch_in(orth_scale_kernel<1>, p, s);
}
template <bool A_MN, bool B_MN, class Epi>
static cudaError_t launch_tiles(bool half, ProductParams& p, const typename Epi::Params& e, cudaStream_t s) {
  return half ? launch_product<false, A_MN, B_MN, Epi>(p, e, s) : launch_product<true, A_MN, B_MN, Epi>(p, e, s);
}

template <bool FINE>
cudaError_t launch_orth_gram(bool half, bool mn, ProductParams& p, const typename SymEpi<false, FINE>::Params& e, cudaStream_t s) {
  return mn ? launch_tiles<true, true, SymEpi<false, FINE>>(half, p, e, s)
            : launch_tiles<false, false, SymEpi<false, FINE>>(half, p, e, s);
}
cudaError_t launch_orth_sums(bool half, bool mn, ProductParams& p, const SumEpi::Params& e, cudaStream_t s) {
  return mn ? launch_tiles<true, true, SumEpi>(half, p, e, s) : launch_tiles<false, false, SumEpi>(half, p, e, s);
}
cudaError_t launch_orth_join(const OrthJoinParams& p, int B, cudaStream_t s) {
  return launch_grid(orth_join_kernel, dim3(p.patches * (p.patches + 1) / 2, B, 1), 256, s, p);
}
template <bool FINE>
cudaError_t launch_orth_poly(bool half, ProductParams& p, const typename SymEpi<true, FINE>::Params& e, cudaStream_t s) {
  return launch_tiles<false, false, SymEpi<true, FINE>>(half, p, e, s);
}
template cudaError_t launch_orth_gram<false>(bool, bool, ProductParams&, const SymEpi<false, false>::Params&, cudaStream_t);
template cudaError_t launch_orth_gram<true>(bool, bool, ProductParams&, const SymEpi<false, true>::Params&, cudaStream_t);
template cudaError_t launch_orth_poly<false>(bool, ProductParams&, const SymEpi<true, false>::Params&, cudaStream_t);
template cudaError_t launch_orth_poly<true>(bool, ProductParams&, const SymEpi<true, true>::Params&, cudaStream_t);
cudaError_t launch_orth_step(bool half, bool mn, ProductParams& p, const StepEpi<false>::Params& e, cudaStream_t s) {
  return mn ? launch_tiles<false, true, StepEpi<false>>(half, p, e, s) : launch_tiles<false, false, StepEpi<false>>(half, p, e, s);
}
cudaError_t launch_orth_last(bool half, bool mn, ProductParams& p, const StepEpi<true>::Params& e, cudaStream_t s) {
  return mn ? launch_tiles<false, true, StepEpi<true>>(half, p, e, s) : launch_tiles<false, false, StepEpi<true>>(half, p, e, s);
}

}  // namespace specv
