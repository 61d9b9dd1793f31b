// Distillation from a teacher's top logits: loss, statistics and gradient.
//
// Row n has K teacher entries (id_j, t_j), id_j = -1 for none.  With
// p_j = exp(t_j / T - L) (L: the teacher's log-sum-exp, or that of the listed
// entries), q = softmax(z / T), m = sum p_j, s = the listed ids' mass under q:
//   D = sum_j p_j (log p_j - log q(id_j))  [+ r (log r - log(1 - s)), r = 1 - m]
//   T dD/dz_v = alpha q_v                  v not listed
//             = beta q_v - sum_{id_j=v} p_j  v listed
//   alpha = m [- r s / (1 - s)],  beta = alpha [+ r / (1 - s)]
// 1 - s is summed over the logits that are not listed, and beta q - p is taken
// as p (exp(log(beta q / p)) - 1), so neither cancels where the student comes
// close to its teacher.
#pragma once

#include "row_common.cuh"

namespace specv {

struct DistillParams {
  RowSplit sp;
  int32_t N, K;
  const void* z;
  int64_t rs;
  const int32_t* ids;
  const float* tl;
  int64_t ts;           // row stride of ids and tl
  const float* tlse;    // or NULL
  const float* weight;  // or NULL
  const float* gloss;   // backward: upstream gradient per row, or NULL
  double invT;          // 1 / T
  float c;              // log2(e) / T
  int32_t tail;
  float* loss;
  float4* stats;        // (max logit, alpha / sum, log(beta q / p) - (z - t) / T, L), sum =
                        // sum exp((z - max) / T); L NaN: a row without result
  void* grad;
  int64_t grs;
  int32_t galigned;
  int32_t* status;
};

constexpr float kNoTail = 9.5367431640625e-07f;  // 2^-20: a smaller teacher tail counts as none

// p = exp(x) for a double argument, to fp32 accuracy at any |x| (the argument's
// part below fp32 resolution enters to first order).
__device__ __forceinline__ float exp_d(double x) {
  const float hi = static_cast<float>(x);
  return hi > -200.f ? expf(hi) * (1.f + static_cast<float>(x - static_cast<double>(hi))) : 0.f;
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

// VW gradient values from element i on, clipped to V.  Each is rounded once,
// to nearest, to the logits' type.
template <int DT>
__device__ __forceinline__ void store_vec(void* row, int64_t i, int64_t V, bool aligned,
                                          const float (&x)[Elem<DT>::VW]) {
  using E = Elem<DT>;
  if (aligned && i + E::VW <= V) {
    uint4 w;
    if (DT == 0) {
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(x[1]), "f"(x[0]));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(x[3]), "f"(x[2]));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.z) : "f"(x[5 % E::VW]), "f"(x[4 % E::VW]));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.w) : "f"(x[7 % E::VW]), "f"(x[6 % E::VW]));
    } else {
      w = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                     __float_as_uint(x[3]));
    }
    *reinterpret_cast<uint4*>(reinterpret_cast<char*>(row) + i * E::ES) = w;
    return;
  }
#pragma unroll
  for (int k = 0; k < E::VW; ++k)
    if (i + k < V) store_elem<DT>(row, i + k, x[k]);
}

// beta q - p at a listed id: z its logit, t and p those of its entry, ps the
// sum of p over its entries, d = log(beta q / p) - (z - t) / T, bq = beta q to
// fp32's accuracy.
__device__ __forceinline__ float listed_grad(float z, float t, float p, float ps, double invT, double d, float bq) {
  if (p > 0.f && ps == p)
    return p * expm1f(static_cast<float>((static_cast<double>(z) - static_cast<double>(t)) * invT + d));
  return bq - ps;
}

// For teacher entry j of a row (ids, p in shared memory): the sum of p over
// entries of the same id, and whether j is the first of them.  Whole warp.
__device__ __forceinline__ float same_id(const int32_t* ids, const float* p, int K, int j, int lane,
                                         bool& first) {
  const int id = ids[j];
  float s = 0.f;
  bool earlier = false;
  for (int i = lane; i < K; i += 32)
    if (ids[i] == id) {
      s += p[i];
      earlier |= i < j;
    }
  first = !__any_sync(0xffffffffu, earlier);
  return warp_sum_f(s);
}

// Block-wide sum of entries of size up to about 1 (threads from K on hold
// none), exact in units of 2^-40: fp64 sums would cost a block microseconds.
__device__ __forceinline__ uint64_t block_sum_fixed(float x, int K, uint64_t* scratch) {
  uint64_t v = 0;
  if ((threadIdx.x & ~31u) < static_cast<unsigned>(K)) {
    v = __float2ull_rn(x * 1099511627776.f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kRowWarps; ++w) v += scratch[w];
  return v;
}
constexpr double kFixedUnit = 9.094947017729282e-13;  // 2^-40

__device__ __forceinline__ float block_max_nan(float x, float* scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
  __syncthreads();
  float m = scratch[0];
#pragma unroll
  for (int w = 1; w < kRowWarps; ++w) m = max_nan(m, scratch[w]);
  return m;
}

struct DistillPart {  // one CTA's share of a row
  float m, rest, listed;
  int32_t bad;
  double a;
};

// Loss, statistics and (grad given) the gradient of the rows: a cluster per row.
template <int DT>
__global__ void __launch_bounds__(kRowThreads, 2) distill_kernel(const DistillParams P) {
  using E = Elem<DT>;
  extern __shared__ __align__(16) char smem[];
  __shared__ uint64_t bars[kRowWarps];
  __shared__ float fred[kRowWarps];
  __shared__ double dred[kRowWarps];
  __shared__ uint64_t ured[kRowWarps];
  __shared__ float rred[kRowWarps], lred[kRowWarps];
  __shared__ double row_L;
  __shared__ DistillPart part[kMaxCluster];
  __shared__ int badbits, row_dead;
  __shared__ float row_max, row_alpha, row_beta;
  __shared__ double row_delta;
  const int C = P.sp.C, K = P.K, V = P.sp.V;
  const int rank = cluster_rank();
  const int64_t row = blockIdx.x / C;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  cluster_arrive();  // waited for before the first remote write
  if (threadIdx.x == 0) badbits = 0;
  RowSlice<DT> sl;
  sl.init(smem, P.sp, rank);
  const char* zrow = reinterpret_cast<const char*>(P.z) + row * P.rs * E::ES;
  char* grow = reinterpret_cast<char*>(P.grad) + row * P.grs * E::ES;
  const float wt = P.weight ? P.weight[row] : 1.f;
  const bool skip = wt == 0.f;
  if (!skip) sl.load(zrow, P.sp, &bars[warp]);

  int32_t* ids = reinterpret_cast<int32_t*>(smem + static_cast<size_t>(P.sp.svec) * 16);
  float* tl = reinterpret_cast<float*>(ids + K);
  float* pj = tl + K;
  float* zj = pj + K;
  float* sj = zj + K;  // p of the entry's id, or -1: not its first entry
  const double invT = P.invT;
  const float c = P.c;
  int bad = 0;
  double L = 0;
  uint64_t mass = 0;  // sum of p, in units of 2^-40
  if (!skip) {
    // the teacher's entries, in every CTA
    float tmax = neg_inf();
    for (int j = threadIdx.x; j < K; j += kRowThreads) {
      const int id = P.ids[row * P.ts + j];
      const float t = P.tl[row * P.ts + j];
      if (id < -1 || id >= V) bad |= kBadToken;
      const bool there = id >= 0 && id < V;
      ids[j] = there ? id : -1;
      tl[j] = there ? t : neg_inf();
      if (there) tmax = max_nan(tmax, t);
    }
    tmax = block_max_nan(tmax, fred);
    if (!(tmax < pos_inf())) bad |= kNonFinite;  // NaN or +inf
    if (P.tlse) {
      L = P.tlse[row];
      if (!isfinite(L)) bad |= kNonFinite;
    } else if (tmax > neg_inf()) {
      float s = 0;
      for (int j = threadIdx.x; j < K; j += kRowThreads)
        s += exp_d((static_cast<double>(tl[j]) - static_cast<double>(tmax)) * invT);
      const uint64_t all = block_sum_fixed(s, K, ured);
      if (threadIdx.x == 0) row_L = static_cast<double>(tmax) * invT + log(static_cast<double>(all) * kFixedUnit);
      __syncthreads();
      L = row_L;
    }
    float p_sum = 0.f;
    for (int j = threadIdx.x; j < K; j += kRowThreads) {
      const float p = tl[j] > neg_inf() ? exp_d(static_cast<double>(tl[j]) * invT - L) : 0.f;
      pj[j] = p;
      p_sum += p;
    }
    mass = block_sum_fixed(fminf(p_sum, 1e6f), K, ured);  // (also: ids and pj are in place)
    if (!sl.load_wait(&bars[warp])) bad |= kTimeout;
  }
  const float mc = block_max_nan(skip ? 0.f : sl.warp_max(), fred);
  // The listed ids of this slice, a warp for each: logits kept apart, and the
  // share of the loss that needs no normaliser.
  double a = 0;
  const int lo = static_cast<int>(sl.base), hi = lo + P.sp.svec * E::VW;
  char* slice = smem;
  auto elem = [&](int i) {
    return DT == 0 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<unsigned short*>(slice)[i - lo]) << 16)
                   : reinterpret_cast<float*>(slice)[i - lo];
  };
  if (!skip) {
    for (int j = warp; j < K; j += kRowWarps) {
      const int id = ids[j];
      if (id < lo || id >= hi) continue;
      const float z = elem(id);
      bool first;
      const float ps = same_id(ids, pj, K, j, lane, first);
      __syncwarp();
      if (lane == 0) {
        if (pj[j] > 0.f)
          a += static_cast<double>(pj[j]) * ((static_cast<double>(tl[j]) - static_cast<double>(z)) * invT - L);
        zj[j] = z;
        sj[j] = first ? ps : -1.f;
      }
    }
  }
  __syncthreads();
  float listed = 0.f, rest = 0.f;
  const float mref = mc > neg_inf() ? mc : 0.f;
  if (!skip) {
    for (int j = warp * 32 + lane; j < K; j += kRowThreads) {
      const int id = ids[j];
      if (id < lo || id >= hi || sj[j] < 0.f) continue;
      listed += ex2((zj[j] - mref) * c);
      if (DT == 0) reinterpret_cast<unsigned short*>(slice)[id - lo] = Elem<0>::neg_inf_raw();
      else reinterpret_cast<float*>(slice)[id - lo] = neg_inf();
    }
  }
  __syncthreads();
  if (!skip) sl.each([&](float z, int) { rest += ex2((z - mref) * c); });
  if (bad) atomicOr(&badbits, bad);
  rest = warp_sum_f(rest);
  listed = warp_sum_f(listed);
  if (lane == 0) {
    rred[warp] = rest;
    lred[warp] = listed;
    dred[warp] = a;
  }
  __syncthreads();
  cluster_wait();
  if (static_cast<int>(threadIdx.x) < C) {
    DistillPart mine;
    mine.m = mc;
    mine.rest = mine.listed = 0.f;
    mine.a = 0;
    mine.bad = badbits;
    for (int w = 0; w < kRowWarps; ++w) {
      mine.rest += rred[w];
      mine.listed += lred[w];
      mine.a += dred[w];
    }
    *peer(part + rank, static_cast<int>(threadIdx.x)) = mine;
  }
  cluster_sync();

  if (threadIdx.x == 0) {  // the row's scalars, once per CTA (64-bit arithmetic is slow)
    float mx = neg_inf();
    int anybad = 0;
    for (int r = 0; r < C; ++r) {
      mx = max_nan(mx, part[r].m);
      anybad |= part[r].bad;
    }
    const bool finite = mx > neg_inf() && mx < pos_inf();
    double S_rest = 0, S_listed = 0, A = 0;
    for (int r = 0; r < C; ++r) {
      const double f = finite ? ex2((part[r].m - mx) * c) : 0.f;
      S_rest += f * part[r].rest;
      S_listed += f * part[r].listed;
      A += part[r].a;
    }
    const bool dead = skip || anybad || !finite;
    const double m = static_cast<double>(mass) * kFixedUnit;
    const double total = S_rest + S_listed;
    const double r = P.tail ? (1.0 - m < kNoTail ? 0.0 : 1.0 - m) : 0.0;
    double alpha = m, beta = m;
    const bool has_rest = S_rest > 0;
    if (r > 0 && has_rest) {
      alpha = m - r * S_listed / S_rest;
      beta = alpha + r * total / S_rest;
    }
    const double lz = static_cast<double>(mx) * invT + log(total);
    row_dead = dead;
    row_max = mx;
    row_alpha = static_cast<float>(alpha / total);
    row_beta = static_cast<float>(beta / total);
    row_delta = log(beta) - lz + L;
    if (rank == 0) {
      double loss = 0;
      if (!dead) {
        loss = A + m * lz;
        if (r > 0) loss += has_rest ? r * (log(r) - log(S_rest / total)) : static_cast<double>(pos_inf());
      }
      P.loss[row] = dead ? 0.f : wt * static_cast<float>(loss);
      if (P.stats)
        P.stats[row] = dead ? make_float4(0.f, 0.f, 0.f, __int_as_float(0x7fc00000))
                            : make_float4(mx, row_alpha, static_cast<float>(row_delta), static_cast<float>(L));
      if (P.status) P.status[row] = skip ? 0 : (anybad | (finite ? 0 : kNonFinite));
    }
  }
  if (!P.grad) return;
  __syncthreads();
  const bool dead = row_dead;
  const float mx = row_max;
  const float f = static_cast<float>(wt * invT);
  const float ga = f * row_alpha;
  for (int j = lane; j < sl.nv; j += 32) {
    float z[E::VW];
    if (dead) {
#pragma unroll
      for (int k = 0; k < E::VW; ++k) z[k] = 0.f;
    } else {
      E::unpack(sl.data[sl.v0 + j], z);
#pragma unroll
      for (int k = 0; k < E::VW; ++k) z[k] = ga * ex2((z[k] - mx) * c);
    }
    store_vec<DT>(grow, sl.base + static_cast<int64_t>(sl.v0 + j) * E::VW, V, P.galigned, z);
  }
  if (dead) return;
  __syncthreads();  // the listed ids' gradients go over what was just written
  for (int j = threadIdx.x; j < K; j += kRowThreads) {
    const int id = ids[j];
    if (id < lo || id >= hi || sj[j] < 0.f) continue;
    store_elem<DT>(grow, id, f * listed_grad(zj[j], tl[j], pj[j], sj[j], invT, row_delta,
                                             row_beta * ex2((zj[j] - mx) * c)));
  }
}

// The gradient from the statistics of an earlier distill_kernel: one pass,
// kBackVecs vectors per thread, a CTA per chunk of a row.
constexpr int kBackVecs = 4;

template <int DT>
__global__ void __launch_bounds__(kRowThreads) distill_backward_kernel(const DistillParams P, int chunks) {
  using E = Elem<DT>;
  extern __shared__ __align__(16) char smem[];
  const int64_t row = blockIdx.x / chunks;
  const int chunk = blockIdx.x % chunks;
  const int K = P.K, V = P.sp.V;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const char* zrow = reinterpret_cast<const char*>(P.z) + row * P.rs * E::ES;
  char* grow = reinterpret_cast<char*>(P.grad) + row * P.grs * E::ES;
  int32_t* ids = reinterpret_cast<int32_t*>(smem);
  float* pj = reinterpret_cast<float*>(ids + K);
  float* tl = pj + K;
  const float4 st = P.stats[row];
  const float wt = (P.weight ? P.weight[row] : 1.f);
  const float up = P.gloss ? P.gloss[row] : 1.f;
  const bool dead = wt == 0.f || st.w != st.w;
  const double invT = P.invT;
  const float c = P.c;
  const float f = dead ? 0.f : static_cast<float>(wt * static_cast<double>(up) * invT);
  const float ga = f * st.y;
  const int64_t i0 = static_cast<int64_t>(chunk) * kRowThreads * kBackVecs * E::VW;
  const int64_t i1 = min(static_cast<int64_t>(V), i0 + static_cast<int64_t>(kRowThreads) * kBackVecs * E::VW);
  typename E::Vec v[kBackVecs];
  if (!dead) {
#pragma unroll
    for (int k = 0; k < kBackVecs; ++k) {
      const int64_t i = i0 + (static_cast<int64_t>(k) * kRowThreads + threadIdx.x) * E::VW;
      if (i < i1) v[k] = (P.sp.aligned && i + E::VW <= V) ? E::vec(zrow, i) : E::gather(zrow, i, V);
    }
    const double L = P.tlse ? static_cast<double>(P.tlse[row]) : static_cast<double>(st.w);
    for (int j = threadIdx.x; j < K; j += kRowThreads) {
      const int id = P.ids[row * P.ts + j];
      const float t = P.tl[row * P.ts + j];
      ids[j] = (id >= 0 && id < V) ? id : -1;
      tl[j] = t;
      pj[j] = (id >= 0 && id < V && t > neg_inf()) ? exp_d(static_cast<double>(t) * invT - L) : 0.f;
    }
  }
#pragma unroll
  for (int k = 0; k < kBackVecs; ++k) {
    const int64_t i = i0 + (static_cast<int64_t>(k) * kRowThreads + threadIdx.x) * E::VW;
    if (i >= i1) break;
    float x[E::VW];
    if (dead) {
#pragma unroll
      for (int e = 0; e < E::VW; ++e) x[e] = 0.f;
    } else {
      E::unpack(v[k], x);
#pragma unroll
      for (int e = 0; e < E::VW; ++e) x[e] = ga * ex2((x[e] - st.x) * c);
    }
    store_vec<DT>(grow, i, V, P.galigned, x);
  }
  if (dead) return;
  __syncthreads();
  for (int j = warp; j < K; j += kRowWarps) {
    const int id = ids[j];
    if (id < i0 || id >= i1) continue;
    bool first;
    const float ps = same_id(ids, pj, K, j, lane, first);
    if (lane == 0 && first) {
      const float z = E::scalar(zrow, id);
      const double beta_sum = static_cast<double>(st.z) + static_cast<double>(st.x) * invT - static_cast<double>(st.w);
      store_elem<DT>(grow, id, f * listed_grad(z, tl[j], pj[j], ps, invT, st.z,
                                               expf(static_cast<float>(beta_sum)) * ex2((z - st.x) * c)));
    }
  }
}

}  // namespace specv
