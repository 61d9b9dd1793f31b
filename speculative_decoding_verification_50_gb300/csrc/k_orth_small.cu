// Small orthogonalised updates in one kernel.
#include "orth_launch.cuh"
#include "orth_small.cuh"
#include "orth_squares.cuh"
#include "product_launch.cuh"

namespace specv {

namespace {

// Descriptor of 16 of K: of a K-major operand (k-th 16 columns), and of an MN-major one
// (k-th 16 rows; its groups of 64 columns are a panel apart).
__device__ __forceinline__ uint64_t small_desc_k(uint32_t plane, int k) {
  return operand_desc<false>(plane + (k >> 2) * (kPlane / 2) + (k & 3) * 32);
}
__device__ __forceinline__ uint64_t small_desc_mn(uint32_t plane, int k) {
  constexpr uint64_t lead = (kPlane / 2) >> 4, stride = 1024 >> 4;
  return ((static_cast<uint64_t>(plane + k * 2048) >> 4) & 0x3fff) | (lead << 16) | (stride << 32) | (1ull << 46) | (2ull << 61);
}

// A B^T of 128 x 128 matrices of three parts, issued by one thread: blocks of 16 of K.  Its
// end arrives on `done`.
template <bool B_MN>
__device__ __forceinline__ void small_product(uint64_t* done, uint32_t tmem, uint32_t a, uint32_t b, int blocks) {
  constexpr uint32_t idesc = (1u << 4) | (B_MN ? 1u << 16 : 0u) | ((kSmallSide >> 3) << 17) | ((kSmallSide >> 4) << 24);
  for (int part = 0; part < 3; ++part) {
    const uint32_t pa = a + (part == 2 ? kPlane : 0), pb = b + (part == 1 ? kPlane : 0);
    for (int k = 0; k < blocks; ++k)
      tc_mma<false>(tmem, small_desc_k(pa, k), B_MN ? small_desc_mn(pb, k) : small_desc_k(pb, k), idesc, part > 0 || k > 0);
  }
  tc_commit<false>(smem_u32(done));
}

// A wait that ran out goes on a little (half a second), so that what products in flight read and
// write is not used again; once one of these ran out too (*gone is 2) they do not.
__device__ __forceinline__ bool small_last_wait(uint64_t* bar, uint32_t parity, volatile int* gone) {
  const long long t0 = clock64();
  do {
    if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
  } while (*gone != 2 && clock64() - t0 < 1000000000LL);
  *gone = 2;
  return false;
}

}  // namespace

template <int DT, int C>
__global__ void __launch_bounds__(kSmallThreads, 1) orth_small_kernel(const __grid_constant__ SmallParams p) {
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t done;
  __shared__ uint32_t tmem_at;
  __shared__ int gone_flag;
  __shared__ ScaledSquares warps[kSmallThreads / 32], mine;
  uint8_t* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint8_t *y = base, *sq = base + 2 * kPlane, *sums = base + 4 * kPlane;  // (high, then low); sums: fp32, or P
  const uint32_t y_at = smem_u32(y), s_at = smem_u32(sq), sum_at = smem_u32(sums);
  volatile int* gone = &gone_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank()), z = blockIdx.x / C;
  const int t0 = rank * kSmallSide;
  if (threadIdx.x == 0) {
    mbar_init(&done, p.stall == z + 1 && rank == 0 ? 2 : 1);
    fence_mbar_init();
    gone_flag = 0;
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 128;" ::"r"(smem_u32(&tmem_at)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait_primary();
  pdl_launch_dependents();

  // The update's 128 x 128 elements of this CTA: a warp reads a row at a time, a lane four
  // of its elements.  r, c: row and column within them as they lie in the update.
  constexpr int ES = Elem<DT>::ES;
  const int rows = p.tall ? min(p.t - t0, kSmallSide) : p.s, cols = p.tall ? p.s : min(p.t - t0, kSmallSide);
  const char* in = static_cast<const char*>(p.in) + (z * p.batch_stride + (p.tall ? t0 * p.row_stride : t0)) * ES;
  float v[16][4];
  ScaledSquares a = {kSquaresLeast, 0.f};
  float inv_m = 1.f / kSquaresLeast;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = 8 * i + warp, c = 4 * lane;
    const char* row = in + r * p.row_stride * ES;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[i][k] = 0.f;
    if (r < rows && c < cols) {
      if (p.vec && c + 4 <= cols) {
        if (DT == 0) {
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(row + c * ES));
          v[i][0] = __uint_as_float(w.x << 16), v[i][1] = __uint_as_float(w.x & 0xffff0000u);
          v[i][2] = __uint_as_float(w.y << 16), v[i][3] = __uint_as_float(w.y & 0xffff0000u);
        } else {
          const float4 w = __ldg(reinterpret_cast<const float4*>(row + c * ES));
          v[i][0] = w.x, v[i][1] = w.y, v[i][2] = w.z, v[i][3] = w.w;
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (c + k < cols) v[i][k] = Elem<DT>::scalar(row, c + k);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) squares_add<4>(a, inv_m, v[i]);
  squares_cta(a, warps, mine);
  cluster_sync();
  ScaledSquares sum = {kSquaresLeast, 0.f};
  for (int q = 0; q < C; ++q) {
    ScaledSquares o;
    const uint32_t from = in_cta(smem_u32(&mine), q);
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o.m) : "r"(from) : "memory");
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o.s) : "r"(from + 4) : "memory");
    squares_join(sum, o);
  }
  const float root = sqrtf(sum.s), inv = 1.f / sum.m;
  const bool bad = !(sum.s < pos_inf());
  const float f = bad || sum.s == 0.f ? 0.f : p.scale / root;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = 8 * i + warp, c = 4 * lane;
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float x0 = bad ? 0.f : v[i][2 * k] * inv * f, x1 = bad ? 0.f : v[i][2 * k + 1] * inv * f;
      hi[k] = pack_f16(x0, x1);
      const float2 g = unpack_f16(hi[k]);
      lo[k] = pack_f16(x0 - g.x, x1 - g.y);
    }
    if (!p.tall) {
      *reinterpret_cast<uint2*>(y + small_at(r, c)) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(y + kPlane + small_at(r, c)) = make_uint2(lo[0], lo[1]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        *reinterpret_cast<uint16_t*>(y + small_at(c + k, r)) = static_cast<uint16_t>(hi[k >> 1] >> (16 * (k & 1)));
        *reinterpret_cast<uint16_t*>(y + kPlane + small_at(c + k, r)) = static_cast<uint16_t>(lo[k >> 1] >> (16 * (k & 1)));
      }
    }
  }
  tc_fence_before();
  fence_async_shared();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;

  // This thread's row and 64 columns (a panel) of a product.
  const int row = (warp & 3) * 32 + lane, panel = warp >> 2;
  const uint32_t mine_at = tmem + panel * 64 + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  const int blocks_s = (p.s + 15) / 16;
  uint32_t phase = 0;
  // Products are issued by thread 0, and waited for by all.  Where one does not end in time no
  // more are issued (lost), and the CTA goes on to the end, for the cluster's barriers.
  bool lost = false;
  auto finish = [&] {
    if (!prod_wait(&done, phase, gone)) lost |= !small_last_wait(&done, phase, gone);
    phase ^= 1;
    __syncwarp();
    tc_fence_after();
  };
  auto ready = [&] {  // what threads wrote to shared memory and read of tensor memory, for products
    tc_fence_before();
    fence_async_shared();
    __syncthreads();
    tc_fence_after();
  };
  for (int k = 0; k < p.steps; ++k) {
    const SmallStep st = p.step[k];
    // S: this CTA's part, then this CTA's rows over all parts
    if (threadIdx.x == 0 && !lost) small_product<false>(&done, tmem, y_at, y_at, kSmallSide / 16);
    finish();
#pragma unroll
    for (int c = 0; c < 64; c += 32) {
      float x[32];
      tmem_load32(mine_at + c, x);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<float4*>(sums + small_sum_at(row, (panel * 64 + c) / 4 + j)) =
            make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    // (16 / C words of this CTA's rows per thread, 16 loads in flight)
    constexpr int kShare = kSmallSide / C, kItems = kShare * 32 / kSmallThreads;
    float4 part[kItems][C];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int r = rank * kShare + 8 * i + warp;
#pragma unroll
      for (int q = 0; q < C; ++q) part[i][q] = load_cluster(in_cta(sum_at + small_sum_at(r, lane), q));
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      float4 x = part[i][0];
#pragma unroll
      for (int q = 1; q < C; ++q) x.x += part[i][q].x, x.y += part[i][q].y, x.z += part[i][q].z, x.w += part[i][q].w;
      x.x *= st.gram, x.y *= st.gram, x.z *= st.gram, x.w *= st.gram;
      const uint32_t h0 = pack_f16(x.x, x.y), h1 = pack_f16(x.z, x.w);
      const float2 g0 = unpack_f16(h0), g1 = unpack_f16(h1);
      const uint32_t l0 = pack_f16(x.x - g0.x, x.y - g0.y), l1 = pack_f16(x.z - g1.x, x.w - g1.y);
      const uint32_t to = s_at + small_at(rank * kShare + 8 * i + warp, 4 * lane);
#pragma unroll
      for (int q = 0; q < C; ++q) {
        store_cluster(in_cta(to, q), h0, h1);
        store_cluster(in_cta(to + kPlane, q), l0, l1);
      }
    }
    asm volatile("fence.proxy.async;" ::: "memory");
    cluster_sync();
    ready();
    // P = b S + c S S, in the place of the sums
    if (threadIdx.x == 0 && !lost) small_product<false>(&done, tmem, s_at, s_at, blocks_s);
    finish();
    auto update = [&](const uint8_t* from, uint8_t* to, float alpha, float beta, bool last) {
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        float x[32];
        tmem_load32(mine_at + c, x);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t at = small_at(row, panel * 64 + c + 8 * j);
          const uint4 h = *reinterpret_cast<const uint4*>(from + at), l = *reinterpret_cast<const uint4*>(from + kPlane + at);
          uint32_t wh[4] = {h.x, h.y, h.z, h.w}, wl[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 g = unpack_f16(wh[i]), d = unpack_f16(wl[i]);
            const float x0 = fmaf(g.x + d.x, beta, x[8 * j + 2 * i] * alpha), x1 = fmaf(g.y + d.y, beta, x[8 * j + 2 * i + 1] * alpha);
            if (last) {
              wh[i] = pack_bf16(x0, x1);
            } else {
              wh[i] = pack_f16(x0, x1);
              const float2 o = unpack_f16(wh[i]);
              wl[i] = pack_f16(x0 - o.x, x1 - o.y);
            }
          }
          *reinterpret_cast<uint4*>(to + at) = make_uint4(wh[0], wh[1], wh[2], wh[3]);
          if (!last) *reinterpret_cast<uint4*>(to + kPlane + at) = make_uint4(wl[0], wl[1], wl[2], wl[3]);
        }
      }
    };
    update(sq, sums, st.poly, st.poly_s, false);
    ready();
    // Y <- a Y + P Y
    if (threadIdx.x == 0 && !lost) small_product<true>(&done, tmem, sum_at, y_at, blocks_s);
    finish();
    update(y, y, st.step, st.step_y, k + 1 == p.steps);
    ready();
  }

  // bf16, from y
  uint16_t* out = p.out + z * p.out_batch_stride + (p.tall ? t0 * p.out_row_stride : t0);
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int r = 8 * i + warp, c = 4 * lane;
    if (r >= rows || c >= cols) continue;
    uint2 w;
    if (!p.tall) {
      w = *reinterpret_cast<const uint2*>(y + small_at(r, c));
    } else {
      uint32_t h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = *reinterpret_cast<const uint16_t*>(y + small_at(c + k, r));
      w = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
    }
    uint16_t* to = out + r * p.out_row_stride + c;
    if (p.out_vec && c + 4 <= cols) {
      *reinterpret_cast<uint2*>(to) = w;
    } else {
      to[0] = static_cast<uint16_t>(w.x);
      if (c + 1 < cols) to[1] = static_cast<uint16_t>(w.x >> 16);
      if (c + 2 < cols) to[2] = static_cast<uint16_t>(w.y);
      if (c + 3 < cols) to[3] = static_cast<uint16_t>(w.y >> 16);
    }
  }
  if (threadIdx.x == 0) {
    if (rank == 0) {
      if (p.norm) p.norm[z] = bad ? __int_as_float(0x7fc00000) : sum.m * root;
      if (p.status) p.status[z] = bad ? kNonFinite : 0;
    }
  }
  __syncthreads();
  cluster_sync();  // (the status is written; and no CTA leaves while others may read of it)
  if (gone_flag && threadIdx.x == 0 && p.status) atomicOr(&p.status[z], kTimeout);
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 128;" ::"r"(tmem) : "memory");
}

template <int DT, int C>
static cudaError_t launch_small(const SmallParams& p, int B, cudaStream_t s) {
  constexpr int kDevices = 64;
  static std::atomic<bool> allowed[kDevices];
  auto kern = orth_small_kernel<DT, C>;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= kDevices || !allowed[dev].load(std::memory_order_acquire)) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmallSmem);
    if (err == cudaSuccess) err = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (err != cudaSuccess) return err;
    if (dev < kDevices) allowed[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(B * C), 1, 1);
  cfg.blockDim = dim3(kSmallThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmallSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int DT>
static cudaError_t launch_small_of(const SmallParams& p, int C, int B, cudaStream_t s) {
  switch (C) {
    case 1: return launch_small<DT, 1>(p, B, s);
    case 2: return launch_small<DT, 2>(p, B, s);
    case 4: return launch_small<DT, 4>(p, B, s);
    case 8: return launch_small<DT, 8>(p, B, s);
    default: return launch_small<DT, 16>(p, B, s);
  }
}

cudaError_t launch_orth_small(int dtype, const SmallParams& p, int C, int B, cudaStream_t s) {
  return dtype == SPECV_BF16 ? launch_small_of<0>(p, C, B, s) : launch_small_of<1>(p, C, B, s);
}

}  // namespace specv
