// Rows of logits held on chip by a thread-block cluster.
//
// The kernels of filtered sampling, of the top logits and of the distillation
// loss need several passes over a row (its maximum, a histogram, a cut, a
// result).  A cluster of C CTAs takes one row: each CTA copies its slice into
// shared memory once (one bulk copy per warp's segment) and every pass after
// that reads shared memory, so HBM sees each logit once.  CTAs exchange a few
// values through distributed shared memory between cluster barriers.
#pragma once

#include "specv_common.cuh"

namespace specv {

constexpr int kRowThreads = 512;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxSegs = kMaxCluster * kRowWarps;

// How a row is spread: CTA r holds vectors [r * svec, (r + 1) * svec) of 16
// bytes, its warp w the segment [w * gvec, (w + 1) * gvec) of them.  Index
// order is (CTA, warp, vector), lanes taking the vectors of a segment in turn.
struct RowSplit {
  int32_t V;
  int32_t C;       // CTAs per row
  int32_t svec;    // vectors per CTA
  int32_t gvec;    // vectors per warp segment
  int32_t aligned; // rows start 16-byte aligned: bulk copies
};

__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}

// The address, in CTA `rank` of the cluster, of this CTA's shared variable p.
template <typename T>
__device__ __forceinline__ T* peer(T* p, int rank) {
  return cg::this_cluster().map_shared_rank(p, rank);
}

__device__ __forceinline__ double warp_sum_d(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float warp_sum_f(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// max of two, NaN if either is NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// One CTA's slice of a row.
template <int DT>
struct RowSlice {
  using E = Elem<DT>;
  using Vec = typename E::Vec;
  Vec* data;      // shared memory, svec vectors
  int v0;         // the segment's first vector, within the slice
  int nv;         // its vectors
  int64_t base;   // index of the slice's first logit in the row
  int lane;

  __device__ void init(char* smem, const RowSplit& sp, int rank) {
    data = reinterpret_cast<Vec*>(smem);
    lane = threadIdx.x & 31;
    const int w = threadIdx.x >> 5;
    const int64_t nvec = (static_cast<int64_t>(sp.V) + E::VW - 1) / E::VW;
    const int64_t first = static_cast<int64_t>(rank) * sp.svec;
    const int mine = static_cast<int>(max(int64_t(0), min(int64_t(sp.svec), nvec - first)));
    v0 = min(w * sp.gvec, mine);
    nv = min((w + 1) * sp.gvec, mine) - v0;
    base = first * E::VW;
  }

  // Starts this warp's copies; load_wait() before the segment is read.  `bar`
  // is the warp's own barrier.
  __device__ void load(const void* row, const RowSplit& sp, uint64_t* bar) {
    const int64_t g0 = base + static_cast<int64_t>(v0) * E::VW;  // the segment's first logit
    if (sp.aligned) {
      const int64_t left = static_cast<int64_t>(sp.V) - g0;
      const int full = static_cast<int>(max(int64_t(0), min(int64_t(nv), left / E::VW)));
      if (lane == 0) {
        mbar_init(bar, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(full) * 16u);
        if (full > 0)
          bulk_load(data + v0, reinterpret_cast<const char*>(row) + g0 * E::ES,
                    static_cast<uint32_t>(full) * 16u, bar);
      }
      // the row's last vector, where V is no multiple of the vector's width
      if (lane == 1 && full < nv) data[v0 + full] = E::gather(row, g0 + int64_t(full) * E::VW, sp.V);
    } else {
      if (lane == 0) {
        mbar_init(bar, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(bar, 0);
      }
      for (int j = lane; j < nv; j += 32) data[v0 + j] = E::gather(row, g0 + int64_t(j) * E::VW, sp.V);
    }
    __syncwarp();
  }

  // False where the copies did not land within the bound (about two seconds).
  __device__ bool load_wait(uint64_t* bar) {
    bool ok = mbar_wait_bounded(bar, 0);
    if (!ok) ok = mbar_wait_bounded(bar, 0);
    __syncwarp();
    return ok;
  }

  // f(z, index) over this lane's logits of the segment, padding (-inf) included.
  template <typename Fn>
  __device__ __forceinline__ void each(Fn&& f) const {
    for (int j = lane; j < nv; j += 32) {
      float z[E::VW];
      E::unpack(data[v0 + j], z);
      const int i0 = static_cast<int>(base) + (v0 + j) * E::VW;
#pragma unroll
      for (int k = 0; k < E::VW; ++k) f(z[k], i0 + k);
    }
  }

  // The maximum over the segment (all lanes), NaN if any logit is NaN.
  __device__ float warp_max() const {
    float m = neg_inf();
    for (int j = lane; j < nv; j += 32) {
      float z[E::VW];
      E::unpack(data[v0 + j], z);
#pragma unroll
      for (int k = 0; k < E::VW; k += 2) m = max3_nan(m, z[k], z[k + 1]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
  }
};

// v into slot[my rank] of every CTA of the cluster (threads 0..C-1 of the CTA
// hold the same v); visible after the next cluster barrier.
template <typename T>
__device__ __forceinline__ void push_all(T* slot, int rank, int C, T v) {
  if (static_cast<int>(threadIdx.x) < C) *peer(slot + rank, static_cast<int>(threadIdx.x)) = v;
}

}  // namespace specv
