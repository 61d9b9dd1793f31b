// Rows of logits over thread-block clusters.
//
// The kernels of filtered sampling, of the top logits and of the distillation
// loss need several passes over a row (its maximum, a histogram, a cut, a
// result).  A cluster of C CTAs takes one row.  Few rows: each CTA copies its
// slice into shared memory once (one bulk copy per warp's segment) and every
// pass reads it there.  Rows enough to fill the SMs: fewer CTAs per row (one or
// two), and every pass streams the slice, the first from HBM and the others mostly
// from L2, so that the fixed costs of a CTA and the waits of a cluster come less
// often per row.  CTAs exchange a few values through distributed shared memory
// between cluster barriers.
#pragma once

#include "specv_common.cuh"

namespace specv {

constexpr int kRowThreads = 512;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kStage = 64;     // vectors of a ring's stage: two per lane
constexpr int kMaxRing = 6;

// Bytes of a CTA's held vectors and its warps' rings.  (From a multiple of 128 bytes
// on: 16 past one, loss + gradient of 1024 x 152064 fp32 take 8 % longer.)
__host__ __device__ constexpr size_t row_bytes(int rvec, int stages) {
  return static_cast<size_t>(rvec + stages * kStage) * kRowWarps * 16;
}

// How a row is spread, in vectors of 16 bytes from its first logit on: CTA r
// holds vectors [r * svec, (r + 1) * svec), its warp w the segment [w * gvec,
// (w + 1) * gvec) of them (-inf after the row's last logit).  Index order is
// (CTA, warp, vector), lanes taking the vectors of a segment in turn; it does
// not depend on the row's alignment, so neither does any sum.  (It does depend on
// the split: sums of whole numbers are rounded to their unit, others to fp32, part
// by part.)
struct RowSplit {
  int32_t V;
  int32_t C;       // CTAs per row
  int32_t svec;    // vectors per CTA
  int32_t gvec;    // vectors per warp segment
  int32_t rvec;    // of them, those held in shared memory (the first)
  int32_t stages;  // of the ring that the others are streamed through, kStage vectors each; 0: plain loads
  int32_t H;       // parts of a CTA's slice that are summed apart (1, 2 or 4)
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

// A vector's logits as pairs of fp32 for the paired arithmetic.
template <int DT>
__device__ __forceinline__ void unpack_pairs(const typename Elem<DT>::Vec& v, uint64_t (&z)[Elem<DT>::VW / 2]) {
  float x[Elem<DT>::VW];
  Elem<DT>::unpack(v, x);
#pragma unroll
  for (int k = 0; k < Elem<DT>::VW / 2; ++k) z[k] = f2(x[2 * k], x[2 * k + 1]);
}

// One thread's share of a softmax: its running maximum and the sum of
// 2^((z - run) c) over what it has seen.
struct RunningSum {
  float run = neg_inf(), sum = 0.f;

  // U vectors as pairs, `top` the larger of their maximum and run.
  template <int N>
  __device__ __forceinline__ void add(const uint64_t (&z)[N], float top, float c) {
    const float ref = top > neg_inf() ? top : 0.f;
    sum *= ex2((run - ref) * c);
    run = top;
    const uint64_t r2 = f2(-ref, -ref), c2 = f2(c, c);
    uint64_t t = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float a, b;
      f2_split(f2_mul(f2_add(z[k], r2), c2), a, b);
      t = f2_add(t, f2(ex2(a), ex2(b)));
    }
    float a, b;
    f2_split(t, a, b);
    sum += a + b;
  }
  // The sum relative to m >= run.
  __device__ __forceinline__ float at(float m, float c) const { return sum > 0.f ? sum * ex2((run - m) * c) : 0.f; }
};

// One CTA's slice of a row, as one warp sees it: its segment.  RING: either
// held whole or streamed through the ring; else held in part (or whole) and the
// rest streamed by plain loads.  (The ring pays where a pass is short: with loads,
// loss and gradient of 1024 x 128256 bf16 take 12 % longer than with a ring of 1 KB
// stages.  Sampling's longer passes and its histograms, which leave room for three
// stages, go the other way: with the ring 2304 x 152064 fp32 take 16 % longer, the
// 256 top logits of 2048 x 152064 bf16 24 %.)
// AHEAD: streamed vectors are loaded two by two, the next two while f has two;
// else four at a time.  (By four the 256 top logits of 2048 x 152064 bf16 take 5 %
// longer; sampling, whose passes have no registers to spare, 1 % less, 2304 x 152064
// fp32.)
template <int DT, bool RING, bool AHEAD>
struct RowSlice {
  using E = Elem<DT>;
  using Vec = typename E::Vec;
  Vec* data;        // in shared memory: the held vectors, or the warp's ring
  uint64_t* bars;   // the warp's barriers: one, or one per stage
  const char* src;  // the segment in memory
  int v0;           // the segment's first vector, within the slice
  int nv, rv;       // its vectors; of them, those held
  int base;         // index of the slice's first place in the row
  int left;         // logits of the row from the segment's first on
  int plain;        // vectors that aligned copies bring (none of a row that starts past a 16-byte boundary)
  int mis;          // bytes by which the row starts past one
  int lane;
  int stages;       // 0: held
  int stage;        // the ring's next stage to be read ...
  uint32_t parity;  // ... and its barrier's phase
  bool primed;      // the next pass's first copies are under way
  int until;        // vectors that copies bring in a pass: `plain`, until one is late (none is issued from then on)
  bool late;        // a copy did not land in time

  __device__ void init(char* smem, uint64_t* barriers, const RowSplit& sp, const void* row, int rank, int w) {
    lane = threadIdx.x & 31;
    const int nvec = static_cast<int>((static_cast<int64_t>(sp.V) + E::VW - 1) / E::VW);
    const int first = rank * sp.svec;
    const int mine = max(0, min(sp.svec, nvec - first));
    v0 = min(w * sp.gvec, mine);
    nv = min((w + 1) * sp.gvec, mine) - v0;
    base = first * E::VW;
    rv = min(nv, sp.rvec);
    stages = RING ? sp.stages : 0;
    data = reinterpret_cast<Vec*>(smem) + w * (sp.rvec + stages * kStage);
    bars = barriers + w * kMaxRing;
    left = sp.V - base - v0 * E::VW;
    src = reinterpret_cast<const char*>(row) + static_cast<int64_t>(base + v0 * E::VW) * E::ES;
    mis = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
    plain = mis == 0 ? max(0, min(nv, left / E::VW)) : 0;
    stage = 0;
    parity = 0;
    primed = false;
    until = plain;
    late = false;
  }

  // Vector j of the segment from memory (-inf after the row's last logit).
  // Rows that start past a 16-byte boundary: two aligned vectors, shifted.
  __device__ __forceinline__ Vec fetch(int j) const {
    union {
      Vec v;
      uint4 u;
      typename E::Raw r[E::VW];
    } x;
    const char* at = src + static_cast<int64_t>(j) * 16 - mis;
    // whole, with both aligned vectors inside the row
    if (mis == 0 ? (j + 1) * E::VW <= left
                 : (v0 + j + base > 0 && (j + 1) * E::VW + (16 - mis) / E::ES <= left)) {
      x.u = __ldcg(reinterpret_cast<const uint4*>(at));
      if (mis != 0) x.u = shift_bytes(x.u, __ldcg(reinterpret_cast<const uint4*>(at) + 1), mis);
    } else {
#pragma unroll
      for (int k = 0; k < E::VW; ++k)
        x.r[k] = j * E::VW + k < left ? reinterpret_cast<const typename E::Raw*>(src)[j * E::VW + k] : E::neg_inf_raw();
    }
    return x.v;
  }

  // Vectors j0 + lane and 32 further (-inf past nv), the whole warp.  Inside a
  // row that starts past a 16-byte boundary each lane loads its aligned vector
  // once and takes the bytes of the next from the lane above (6 % of 608 x 152064
  // fp32 top-p, 7 % of loss + gradient of 1024 x 128256 bf16).
  __device__ __forceinline__ void fetch_two(int j0, Vec (&x)[2]) const {
    const int j = j0 + lane;
    if (mis != 0 && v0 + j0 + base > 0 && j0 + kStage <= nv && (j0 + kStage) * E::VW + (16 - mis) / E::ES <= left) {
      x[0] = shifted(j);
      x[1] = shifted(j + 32);
      return;
    }
    x[0] = j < nv ? fetch(j) : none();
    x[1] = j + 32 < nv ? fetch(j + 32) : none();
  }
  __device__ __forceinline__ Vec shifted(int j) const {
    const uint4* at = reinterpret_cast<const uint4*>(src + static_cast<int64_t>(j) * 16 - mis);
    union {
      uint4 u;
      Vec v;
    } a;
    a.u = __ldcg(at);
    uint4 n = a.u;
    if (lane == 31) n = __ldcg(at + 1);
    const uint4 up = make_uint4(__shfl_down_sync(0xffffffffu, a.u.x, 1), __shfl_down_sync(0xffffffffu, a.u.y, 1),
                                __shfl_down_sync(0xffffffffu, a.u.z, 1), __shfl_down_sync(0xffffffffu, a.u.w, 1));
    a.u = shift_bytes(a.u, lane == 31 ? n : up, mis);
    return a.v;
  }

  // Vector j < nv, held or not.
  __device__ __forceinline__ Vec vec(int j) const { return j < rv ? data[j] : fetch(j); }

  __device__ __forceinline__ static Vec none() {
    union {
      typename E::Raw r[E::VW];
      Vec v;
    } x;
#pragma unroll
    for (int k = 0; k < E::VW; ++k) x.r[k] = E::neg_inf_raw();
    return x.v;
  }

  // Lane 0: the segment's vectors from v on into stage s of the ring.
  __device__ __forceinline__ void issue(int v, int s) const {
    const uint32_t bytes = static_cast<uint32_t>(min(kStage, plain - v)) * 16u;
    mbar_arrive_expect_tx(&bars[s], bytes);
    bulk_load(data + s * kStage, src + static_cast<int64_t>(v) * 16, bytes, &bars[s], false);
  }
  // (All lanes: what the last pass read has been used by every lane.)  stall (a
  // test hook): the first stage waits for 16 bytes that no copy brings.
  __device__ void prime(bool stall = false) {
    __syncwarp();
    if (lane == 0 && !late) {
      if (stall) mbar_expect_tx(&bars[stage], 16);
      for (int c = 0; c < stages && c * kStage < plain; ++c) issue(c * kStage, (stage + c) % stages);
    }
    primed = true;
  }

  // Starts this warp's copies.  Held rows that start at a 16-byte boundary take
  // one bulk copy.
  __device__ void load(bool stall = false) {
    if (RING && stages > 0) {
      if (lane == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&bars[s], 1);
        fence_mbar_init();
      }
      __syncwarp();
      prime(stall);
      return;
    }
    if (lane == 0) {
      mbar_init(bars, 1);
      fence_mbar_init();
      if (stall) mbar_expect_tx(bars, 16);
      const uint32_t bytes = static_cast<uint32_t>(min(plain, rv)) * 16u;
      mbar_arrive_expect_tx(bars, bytes);
      if (bytes > 0) bulk_load(data, src, bytes, bars, rv == nv);
    }
    constexpr int U = 4;
    for (int j0 = plain + lane; j0 < rv; j0 += 32 * U) {
      Vec x[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (j0 + 32 * u < rv) x[u] = fetch(j0 + 32 * u);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (j0 + 32 * u < rv) data[j0 + 32 * u] = x[u];
    }
    __syncwarp();
  }

  // A bounded wait (about two seconds) for a pass's copy of the vectors from v on.
  // After a late one only those that have been issued are waited for, then nothing.
  __device__ __forceinline__ void wait(uint64_t* bar, uint32_t phase, int v) {
    if (mbar_try_wait(bar, phase)) return;
    if (late && v >= until) return;
    const long long t0 = clock64();
    for (uint32_t it = 0; it < (1u << 21); ++it) {
      if (mbar_try_wait_sleep(bar, phase, 20000u)) return;
      if (clock64() - t0 > 4000000000LL) break;
    }
    late = true;
    until = min(until, v + (stages - (v > 0)) * kStage);
  }

  // Before held vectors are read for the first time.
  __device__ void ready() {
    if (!RING || stages == 0) {
      wait(bars, 0, 0);
      __syncwarp();
    }
  }

  // f(two vectors 32 apart, number of the first) over this lane's vectors of the
  // segment, -inf past its end.  The whole warp calls f together; j < nv says
  // whether the lane's vectors exist (the second: j + 32 < nv).  first: the
  // pass waits for the held vectors, after those that are streamed.
  template <typename Fn>
  __device__ __forceinline__ void groups(Fn&& f, bool first = false) {
    if (!RING) {
      int j0 = rv;  // (a multiple of kStage, or the segment's end)
      if (!AHEAD) {
#pragma unroll 1
        for (; j0 + 2 * kStage <= plain; j0 += 2 * kStage) {
          const Vec* at = reinterpret_cast<const Vec*>(src) + j0 + lane;
          const Vec x[2] = {at[0], at[32]}, y[2] = {at[64], at[96]};
          f(x, j0 + lane);
          f(y, j0 + lane + kStage);
        }
      } else if (j0 + kStage <= plain) {
        const Vec* at = reinterpret_cast<const Vec*>(src) + j0 + lane;
        Vec x[2] = {at[0], at[32]}, y[2] = {x[0], x[1]};
#pragma unroll 1
        for (;;) {
          const bool more = j0 + 2 * kStage <= plain;
          if (more) y[0] = at[kStage], y[1] = at[kStage + 32];
          f(x, j0 + lane);
          j0 += kStage;
          if (!more) break;
          const bool again = j0 + 2 * kStage <= plain;
          if (again) x[0] = at[2 * kStage], x[1] = at[2 * kStage + 32];
          at += 2 * kStage;
          f(y, j0 + lane);
          j0 += kStage;
          if (!again) break;
        }
      }
#pragma unroll 1
      for (; j0 < nv; j0 += kStage) {
        Vec x[2];
        fetch_two(j0, x);
        f(x, j0 + lane);
      }
    }
    if (first) ready();
    if (!RING || stages == 0) {
#pragma unroll 1
      for (int j0 = 0; j0 < rv; j0 += kStage) {
        const int j = j0 + lane;
        const Vec x[2] = {j < rv ? data[j] : none(), j + 32 < rv ? data[j + 32] : none()};
        f(x, j);
      }
      return;
    }
    int j0 = 0;
    if (!primed) prime();
    primed = false;
#pragma unroll 1
    for (; j0 < plain; j0 += kStage) {
      const int j = j0 + lane;
      wait(&bars[stage], parity, j0);
      const Vec* at = data + stage * kStage + lane;
      Vec x[2] = {at[0], at[32]};
      // Every lane has been through f for the chunk before, so its reads of that
      // stage have ended and it can be filled again.  (Not this chunk's stage:
      // its reads are only under way.  Filled here, a copy from L2 overtook them.)
      __syncwarp();
      if (lane == 0 && j0 > 0 && j0 + (stages - 1) * kStage < until)
        issue(j0 + (stages - 1) * kStage, stage == 0 ? stages - 1 : stage - 1);
      if (++stage == stages) {
        stage = 0;
        parity ^= 1;
      }
      if (j0 + kStage > plain) {  // the segment's last chunk: the rest is read without a copy
        if (j >= plain) x[0] = j < nv ? fetch(j) : none();
        if (j + 32 >= plain) x[1] = j + 32 < nv ? fetch(j + 32) : none();
      }
      f(x, j);
    }
    if (late) until = 0;
#pragma unroll 1
    for (; j0 < nv; j0 += kStage) {
      Vec x[2];
      fetch_two(j0, x);
      f(x, j0 + lane);
    }
  }

  // The q-th of n pieces of warp w's segment, of whole stages.
  __device__ RowSlice piece(char* smem, uint64_t* barriers, const RowSplit& sp, const void* row, int rank, int w, int q,
                            int n) const {
    RowSlice s;
    s.init(smem, barriers, sp, row, rank, w);
    const int per = ((s.nv + n - 1) / n + kStage - 1) / kStage * kStage, at = min(q * per, s.nv);
    s.data += at;
    s.rv = max(0, min(per, s.rv - at));
    s.src += static_cast<int64_t>(at) * 16;
    s.v0 += at;
    s.nv = min(per, s.nv - at);
    s.left -= at * E::VW;
    s.plain = s.mis == 0 ? max(0, min(s.nv, s.left / E::VW)) : 0;
    return s;
  }

  // f(z, index) over this lane's logits of the segment, padding (-inf) included.
  template <typename Fn>
  __device__ __forceinline__ void each(Fn&& f) {
    groups([&](const Vec(&x)[2], int j) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float z[E::VW];
        E::unpack(x[u], z);
        const int i0 = index(j + 32 * u);
#pragma unroll
        for (int k = 0; k < E::VW; ++k) f(z[k], i0 + k);
      }
    });
  }

  // Index in the row of vector j's first logit.
  __device__ __forceinline__ int index(int j) const { return base + (v0 + j) * E::VW; }

  // The maximum over the segment (all lanes), NaN if any logit is NaN; `mine`:
  // over each half of this lane's vectors (in turn); `rs`, if given, gets this
  // lane's running sum on the way.
  __device__ float warp_max(float (&mine)[2], RunningSum* rs = nullptr, float c = 0.f) {
    mine[0] = mine[1] = neg_inf();
    groups([&](const Vec(&x)[2], int) {
#pragma unroll
      for (int u = 0; u < 2; ++u) mine[u] = vec_max<DT>(x[u], mine[u]);
      if (rs) {
        uint64_t z[E::VW], lo[E::VW / 2], hi[E::VW / 2];
        unpack_pairs<DT>(x[0], lo);
        unpack_pairs<DT>(x[1], hi);
#pragma unroll
        for (int k = 0; k < E::VW / 2; ++k) {
          z[k] = lo[k];
          z[E::VW / 2 + k] = hi[k];
        }
        rs->add(z, max_nan(mine[0], mine[1]), c);
      }
    }, true);
    float m = max_nan(mine[0], mine[1]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
  }

  // The row's logit of index i, from memory.
  __device__ __forceinline__ float logit(int i) const {
    return E::scalar(src - static_cast<int64_t>(base + v0 * E::VW) * E::ES, i);
  }

  // Logit k of vector j of the segment.
  __device__ __forceinline__ float at(int j, int k) const {
    typename E::Raw r;
    if (j < rv) r = reinterpret_cast<const typename E::Raw*>(data)[j * E::VW + k];
    else r = j * E::VW + k < left ? reinterpret_cast<const typename E::Raw*>(src)[j * E::VW + k] : E::neg_inf_raw();
    if constexpr (DT == 0) return __uint_as_float(static_cast<uint32_t>(r) << 16);
    else return r;
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
      __stcs(reinterpret_cast<uint4*>(at), w);  // (not read again: rows that are stay in L2)
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
      if (next) __stcs(reinterpret_cast<uint4*>(at + skip), shift_bytes(w, n, skip));
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

// v into slot[my rank] of every CTA of the cluster (threads 0..C-1 of the CTA
// hold the same v); visible after the next cluster barrier.
template <typename T>
__device__ __forceinline__ void push_all(T* slot, int rank, int C, T v) {
  if (static_cast<int>(threadIdx.x) < C) *peer(slot + rank, static_cast<int>(threadIdx.x)) = v;
}

}  // namespace specv
