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

// How a row is spread, in vectors of 16 bytes from its first logit on: CTA r
// holds vectors [r * svec, (r + 1) * svec), its warp w the segment [w * gvec,
// (w + 1) * gvec) of them (-inf after the row's last logit).  Index order is
// (CTA, warp, vector), lanes taking the vectors of a segment in turn; it does
// not depend on the row's alignment, so neither does any sum.
struct RowSplit {
  int32_t V;
  int32_t C;       // CTAs per row
  int32_t svec;    // vectors per CTA
  int32_t gvec;    // vectors per warp segment
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

// Bytes [n, n + 16) of the 32 bytes a, b; 0 < n < 16.
__device__ __forceinline__ uint4 shift_bytes(const uint4& a, const uint4& b, int n) {
  uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  const int bits = (n & 3) * 8;
  if (n & 4) {
#pragma unroll
    for (int q = 0; q < 7; ++q) x[q] = x[q + 1];
  }
  if (n & 8) {
#pragma unroll
    for (int q = 0; q < 6; ++q) x[q] = x[q + 2];
  }
  return make_uint4(__funnelshift_r(x[0], x[1], bits), __funnelshift_r(x[1], x[2], bits),
                    __funnelshift_r(x[2], x[3], bits), __funnelshift_r(x[3], x[4], bits));
}

// The maximum of a vector's logits, NaN if any is (bf16: in pairs).
template <int DT>
__device__ __forceinline__ float vec_max(const typename Elem<DT>::Vec& v, float m) {
  if constexpr (DT == 0) {
    uint32_t a, b;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(v.x), "r"(v.y));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(v.z), "r"(v.w));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
    return max3_nan(m, __uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
  } else {
    return max3_nan(max3_nan(m, v.x, v.y), v.z, v.w);
  }
}

// One CTA's slice of a row.
template <int DT>
struct RowSlice {
  using E = Elem<DT>;
  using Vec = typename E::Vec;
  Vec* data;      // shared memory, svec vectors
  int v0;         // the segment's first vector, within the slice
  int nv;         // its vectors
  int base;       // index of the slice's first place in the row
  int lane;

  __device__ void init(char* smem, const RowSplit& sp, int rank) {
    data = reinterpret_cast<Vec*>(smem);
    lane = threadIdx.x & 31;
    const int w = threadIdx.x >> 5;
    const int nvec = static_cast<int>((static_cast<int64_t>(sp.V) + E::VW - 1) / E::VW);
    const int first = rank * sp.svec;
    const int mine = max(0, min(sp.svec, nvec - first));
    v0 = min(w * sp.gvec, mine);
    nv = min((w + 1) * sp.gvec, mine) - v0;
    base = first * E::VW;
  }

  // Starts this warp's copies; load_wait() before the segment is read.  `bar`
  // is the warp's own barrier.  Rows that start at a 16-byte boundary take one
  // bulk copy; others are loaded in aligned vectors, two for each of the row's,
  // and shifted.
  __device__ void load(const void* row, const RowSplit& sp, uint64_t* bar) {
    const int i0 = base + v0 * E::VW;  // the segment's first logit
    const int full = max(0, min(nv, (sp.V - i0) / E::VW));
    const char* src = reinterpret_cast<const char*>(row) + static_cast<int64_t>(i0) * E::ES;
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
    if (lane == 0) {
      const uint32_t bytes = mis == 0 ? static_cast<uint32_t>(full) * 16u : 0u;
      mbar_init(bar, 1);
      fence_mbar_init();
      mbar_arrive_expect_tx(bar, bytes);
      if (bytes > 0) bulk_load(data + v0, src, bytes, bar);
    }
    if (mis == 0) {
      if (lane == 1 && full < nv) data[v0 + full] = E::gather(row, i0 + full * E::VW, sp.V);
    } else {
      constexpr int U = 4;
      for (int j0 = lane; j0 < nv; j0 += 32 * U) {
        uint4 a[U], b[U];
        bool in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = j0 + 32 * u, i = i0 + j * E::VW;
          // both aligned vectors lie inside the row
          in[u] = j < nv && i * E::ES >= mis && static_cast<int64_t>(i) * E::ES - mis + 32 <= static_cast<int64_t>(sp.V) * E::ES;
          if (in[u]) {
            const uint4* p = reinterpret_cast<const uint4*>(src + static_cast<int64_t>(j) * 16 - mis);
            a[u] = __ldg(p);
            b[u] = __ldg(p + 1);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = j0 + 32 * u;
          if (in[u])
            *reinterpret_cast<uint4*>(data + v0 + j) = shift_bytes(a[u], b[u], mis);
          else if (j < nv)
            data[v0 + j] = E::gather(row, i0 + j * E::VW, sp.V);
        }
      }
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
      const int i0 = base + (v0 + j) * E::VW;
#pragma unroll
      for (int k = 0; k < E::VW; ++k) f(z[k], i0 + k);
    }
  }

  // The maximum over the segment (all lanes), NaN if any logit is NaN; `mine`:
  // over this lane's logits.
  __device__ float warp_max(float& mine) const {
    float m = neg_inf();
#pragma unroll 4
    for (int j = lane; j < nv; j += 32) m = vec_max<DT>(data[v0 + j], m);
    mine = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
  }

  // The logit at place i of the slice.
  __device__ __forceinline__ float at(int i) const {
    if constexpr (DT == 0)
      return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const unsigned short*>(data)[i]) << 16);
    else
      return reinterpret_cast<const float*>(data)[i];
  }
};

// VW values, rounded once to nearest to the logits' type.
template <int DT>
__device__ __forceinline__ uint4 pack_vec(const float (&x)[Elem<DT>::VW]) {
  constexpr int W = Elem<DT>::VW;
  uint4 w;
  if (DT == 0) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(x[1]), "f"(x[0]));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(x[3]), "f"(x[2]));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.z) : "f"(x[5 % W]), "f"(x[4 % W]));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.w) : "f"(x[7 % W]), "f"(x[6 % W]));
  } else {
    w = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  return w;
}

template <int DT>
__device__ __forceinline__ void store_elem(void* row, int64_t i, float x) {
  if (DT == 0) {
    uint32_t h;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(0.f), "f"(x));
    reinterpret_cast<unsigned short*>(row)[i] = static_cast<unsigned short>(h & 0xffffu);
  } else {
    reinterpret_cast<float*>(row)[i] = x;
  }
}

// One warp's store of 32 consecutive vectors (lane l holds w, the values of
// indices i .. i + VW - 1, i rising by VW per lane) to a row of V, whatever its
// alignment: lanes exchange halves so that all but the ends go out as aligned
// 16-byte stores.  `on`: the lane holds a vector.  Whole warp.
template <int DT>
__device__ __forceinline__ void store_warp(void* row, int i, int V, bool on, uint4 w) {
  using E = Elem<DT>;
  char* at = reinterpret_cast<char*>(row) + static_cast<int64_t>(i) * E::ES;
  const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15);  // the same in every lane
  const bool inside = on && i >= 0 && i + E::VW <= V;
  if (mis == 0) {
    if (inside) {
      *reinterpret_cast<uint4*>(at) = w;
      return;
    }
  } else {
    // The aligned vector that starts 16 - mis bytes into this lane's: its
    // bytes [16 - mis, 16), then the next lane's first 16 - mis.
    const int lane = threadIdx.x & 31;
    uint4 n;
    n.x = __shfl_down_sync(0xffffffffu, w.x, 1);
    n.y = __shfl_down_sync(0xffffffffu, w.y, 1);
    n.z = __shfl_down_sync(0xffffffffu, w.z, 1);
    n.w = __shfl_down_sync(0xffffffffu, w.w, 1);
    const bool next = __shfl_down_sync(0xffffffffu, inside, 1) && lane < 31;
    const bool prev = __shfl_up_sync(0xffffffffu, inside, 1) && lane > 0;
    if (inside) {
      const int skip = 16 - mis;
      if (next) *reinterpret_cast<uint4*>(at + skip) = shift_bytes(w, n, skip);
      // what no aligned vector covers: the first lane's head, the last's tail
      const uint32_t own[4] = {w.x, w.y, w.z, w.w};
      const int head = skip / E::ES;
#pragma unroll
      for (int k = 0; k < E::VW; ++k) {
        if (k < head ? prev : next) continue;
        if (DT == 0) reinterpret_cast<unsigned short*>(at)[k] = static_cast<unsigned short>(own[k / 2] >> (k % 2 * 16));
        else reinterpret_cast<uint32_t*>(at)[k] = own[k % 4];
      }
      return;
    }
  }
  if (on) {
    const uint32_t own[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < E::VW; ++k) {
      if (i + k < 0 || i + k >= V) continue;
      if (DT == 0) reinterpret_cast<unsigned short*>(at)[k] = static_cast<unsigned short>(own[k / 2] >> (k % 2 * 16));
      else reinterpret_cast<uint32_t*>(at)[k] = own[k % 4];
    }
  }
}

// A vector's logits as pairs of fp32 for the paired arithmetic.
template <int DT>
__device__ __forceinline__ void unpack_pairs(const typename Elem<DT>::Vec& v, uint64_t (&z)[Elem<DT>::VW / 2]) {
  float x[Elem<DT>::VW];
  Elem<DT>::unpack(v, x);
#pragma unroll
  for (int k = 0; k < Elem<DT>::VW / 2; ++k) z[k] = f2(x[2 * k], x[2 * k + 1]);
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// v into slot[my rank] of every CTA of the cluster (threads 0..C-1 of the CTA
// hold the same v); visible after the next cluster barrier.
template <typename T>
__device__ __forceinline__ void push_all(T* slot, int rank, int C, T v) {
  if (static_cast<int>(threadIdx.x) < C) *peer(slot + rank, static_cast<int>(threadIdx.x)) = v;
}

}  // namespace specv
