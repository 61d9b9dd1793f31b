// Distillation from a teacher's top logits: loss, statistics and gradient.
//
// Row n has K teacher entries (id_j, t_j), id_j = -1 for none.  With
// p_j = exp(t_j / T - L) (L: the teacher's log-sum-exp, or that of the listed
// entries), q = softmax(z / T), m = sum p_j, s = the listed ids' mass under q:
//   D = sum_j p_j (log p_j - log q(id_j))  [+ r (log r - log(1 - s)), r = 1 - m]
//   T dD/dz_v = alpha q_v                  v not listed
//             = beta q_v - sum_{id_j=v} p_j  v listed
//   alpha = m [- r s / (1 - s)],  beta = m [+ r]
// 1 - s is summed over the logits that are not listed, relative to the largest of
// them (they may all lie 100 / T and more below the listed ones, where exp(z - max)
// underflows but neither log(1 - s) nor q / (1 - s) does), and beta q - p is taken
// as p (exp(log(beta q / p)) - 1), so neither cancels where the student comes
// close to its teacher.  The logarithms that the loss and the listed ids' gradients
// are differences of are pairs of fp32 (z / T has thousands of units at low
// temperatures; a loss of 0.01 lies in the last bits of its terms).
//
// All of it in fp32, differences taken before they are scaled; sums of p are
// exact in units of 2^-40.  (An SM does two fp64 operations a clock: a few of
// them per thread took longer than the passes over the row.)
#pragma once

#include "row_common.cuh"
#include "specv_device.cuh"  // FF

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
  float ih, il;         // 1 / T: rounded to fp32, and the rest
  float c;              // log2(e) / T
  int32_t tail;
  float* loss;
  float4* stats;        // (ref, A, max logit, beta / sum), sum = sum exp((z - max) / T),
                        // alpha q_v = A exp((z_v - ref) / T); ref NaN: a row without result
  void* grad;
  int64_t grs;
  int32_t* status;
  int32_t stall[2];     // test hook: 1 + the row whose first, second pass waits in vain
};

constexpr float kNoTail = 9.5367431640625e-07f;  // 2^-20: a smaller teacher tail counts as none
constexpr float kFixed = 1099511627776.f;        // 2^40

// exp(d / T) for d <= about 100, good to fp32's rounding of the result: the
// product's error enters to first order.
__device__ __forceinline__ float exp_over(float d, float ih, float il) {
  const float x = __fmul_rn(d, ih);
  const float e = fmaf(d, il, fmaf(d, ih, -x));
  return x > -100.f ? expf(x) * (1.f + e) : 0.f;
}

// The loss is a small difference of logarithms: the few numbers of a row that it
// depends on are pairs of fp32 (FF).
// Sums of a few terms: the low parts gather what the high parts lose, without
// carries (a chain of ff_add takes three times as long).
__device__ __forceinline__ FF ff_gather(FF x, FF y) {
  const FF v = two_sum(x.hi, y.hi);
  return FF{v.hi, (x.lo + y.lo) + v.lo};
}
__device__ __forceinline__ FF ff_times(FF x, float y) {
  const float p = __fmul_rn(x.hi, y);
  return FF{p, fmaf(x.lo, y, fmaf(x.hi, y, -p))};
}

constexpr float kLn2 = 0.693147182464599609375f, kLn2Rest = -1.904654e-9f;

// log(x): the exponent's part as a pair, the mantissa's (0.7 to 1.4) to 2^-25.
__device__ __forceinline__ FF log_pair(float x) {
  if (!(x >= 1.17549435e-38f && x < pos_inf())) return ff(logf(x));
  const int e = (__float_as_int(x) - 0x3f350000) >> 23;
  const float k = static_cast<float>(e);
  const FF m = ff_mul(k, kLn2);
  return ff_gather(FF{m.hi, fmaf(k, kLn2Rest, m.lo)}, ff(logf(__int_as_float(__float_as_int(x) - (e << 23)))));
}

// exp(x) for x <= 0 (0 below -87): x = k ln 2 + f, and f's series to the 7th power,
// good to about 2^-27.
__device__ __forceinline__ FF exp_pair(FF x) {
  if (!(x.hi > -87.f)) return ff(0.f);
  const float k = rintf(x.hi * 1.44269504f);
  const float f = fmaf(-k, kLn2, x.hi), rest = x.lo - k * kLn2Rest;
  const float q = f * f *
      fmaf(f, fmaf(f, fmaf(f, fmaf(f, fmaf(f, 1.f / 5040, 1.f / 720), 1.f / 120), 1.f / 24), 1.f / 6), 0.5f);
  const FF one = two_sum(1.f, f);
  const float lo = one.lo + q, scale = __int_as_float((static_cast<int>(k) + 127) << 23);
  const FF v = two_sum(one.hi, fmaf(one.hi + lo, rest, lo));
  return FF{v.hi * scale, v.lo * scale};
}

__device__ __forceinline__ float warp_max_nan(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

__device__ __forceinline__ float block_max_nan(float x, float* scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, o));
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
  __syncthreads();
  float m = scratch[0];
#pragma unroll
  for (int w = 1; w < kRowWarps; ++w) m = max_nan(m, scratch[w]);
  return m;
}

// (a - b) / T, to about 2^-45 of it (infinite: as hi alone).
__device__ __forceinline__ FF over(float a, float b, float ih, float il) {
  const FF d = two_sum(a, -b);
  const float hi = __fmul_rn(d.hi, ih);
  return FF{hi, fabsf(hi) < 1e30f ? fmaf(d.lo, ih, fmaf(d.hi, il, fmaf(d.hi, ih, -hi))) : 0.f};
}

// What a CTA knows of a row's teacher.
struct Teacher {
  float L;         // the log-sum-exp that was given
  float tmax;      // without one: the largest entry, and
  float pscale;    //   one by the sum of exp((t - tmax) / T); p_j = pj pscale
  uint64_t mass;   // sum of pj, in units of 2^-40 (where it was asked for)
  int bad;         // this thread's findings

  __device__ __forceinline__ float sum() const { return static_cast<float>(mass) * (1.f / kFixed); }
  // sum of p_j
  __device__ __forceinline__ FF total(bool given) const {
    if (!given) return ff(mass ? 1.f : 0.f);
    const float hi = static_cast<float>(mass);
    return FF{hi * (1.f / kFixed), static_cast<float>(static_cast<int64_t>(mass) - static_cast<int64_t>(hi)) * (1.f / kFixed)};
  }
  // log p_j less t_j / T (tmax / T without a log-sum-exp), as a pair, negated
  __device__ __forceinline__ FF norm(bool given) const { return given ? ff(L) : log_pair(sum()); }
};

// The row's entries into shared memory (ids, -1 where absent; logits, -inf
// there; pj), by the whole CTA.  With MASS it ends with a barrier; without, a
// barrier is left to the caller (where a log-sum-exp is given there is none:
// the backward pass of 1024 x 152064 fp32 is 3 us shorter without).
template <bool MASS>
__device__ Teacher load_teacher(const DistillParams& P, int64_t row, int32_t* ids, float* tl, float* pj, float* fred,
                                uint64_t* ured) {
  const int K = P.K, V = P.sp.V;
  const float ih = P.ih, il = P.il;
  Teacher t = {};
  t.pscale = 1.f;
  bool some = true;  // (without a log-sum-exp: there are entries)
  float mx = neg_inf();
  for (int j = threadIdx.x; j < K; j += kRowThreads) {
    const int id = P.ids[row * P.ts + j];
    const float x = P.tl[row * P.ts + j];
    if (id < -1 || id >= V) t.bad |= kBadToken;
    const bool there = id >= 0 && id < V;
    ids[j] = there ? id : -1;
    tl[j] = there ? x : neg_inf();
    if (there && !(x < pos_inf())) t.bad |= kNonFinite;  // NaN or +inf
    if (there) mx = max_nan(mx, x);
  }
  uint64_t v = 0;
  if (P.tlse) {
    t.L = P.tlse[row];
    if (!isfinite(t.L)) t.bad |= kNonFinite;
    // p = exp(t / T - L); the product's rounding, 0.01 and more where t / T is 10^5,
    // belongs to the argument
    for (int j = threadIdx.x; j < K; j += kRowThreads) {
      const float x = __fmul_rn(tl[j], ih);
      const FF d = two_sum(x - t.L, fmaf(tl[j], il, fmaf(tl[j], ih, -x)));
      const float p = tl[j] > neg_inf() && d.hi > -100.f ? expf(d.hi) * (1.f + d.lo) : 0.f;
      pj[j] = p;
      if (MASS) v += __float2ull_rn(fminf(p, 1e6f) * kFixed);
    }
  } else {  // relative to the largest, normalised by pscale
    t.tmax = block_max_nan(mx, fred);
    some = t.tmax > neg_inf() && t.tmax < pos_inf();
    for (int j = threadIdx.x; j < K; j += kRowThreads) {
      const float e = some && tl[j] > neg_inf() ? exp_over(tl[j] - t.tmax, ih, il) : 0.f;
      pj[j] = e;
      v += __float2ull_rn(e * kFixed);
    }
  }
  if (MASS || !P.tlse) {
    if ((threadIdx.x & ~31u) < static_cast<unsigned>(K)) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    if ((threadIdx.x & 31) == 0) ured[threadIdx.x >> 5] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) t.mass += ured[w];
  }
  if (!P.tlse) t.pscale = some && t.mass ? 1.f / t.sum() : 0.f;
  return t;
}

// beta q - p at a listed id: z its logit, t and p those of its entry, ps the
// sum of p over its entries, b = beta / sum, lb its logarithm, ln the entries'
// normaliser.  Like sizes of the two logarithms are taken apart first.
__device__ __forceinline__ float listed_grad(const DistillParams& P, const Teacher& te, float z, float t, float p,
                                             float ps, float mx, float b, FF lb, FF ln) {
  const FF q = over(z, mx, P.ih, P.il);  // log(beta q) less lb
  const float bq = q.hi > -100.f ? b * (expf(q.hi) * (1.f + q.lo)) : 0.f;
  if (!(p > 0.f && ps == p)) return bq - ps;
  if (!(q.hi > -1e30f)) return -p;
  const FF o = over(t, P.tlse ? 0.f : te.tmax, P.ih, P.il);
  const FF d = ff_gather(ff_gather(q, ff_neg(o)), ff_gather(ln, lb));
  const float x = d.hi + d.lo;
  return x < 1.f ? p * expm1f(x) : bq - p;
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

struct DistillPart {  // a warp's or a CTA's share of a row
  float mr, ml;                // the largest logit that is not listed, and that is
  FF rest, listed;             // sums relative to them
  FF a;
  int32_t bad;
};
constexpr int kRuledOut = 1 << 30;  // among the bad bits: a listed token has mass and no probability

// The sum of n <= 16 parts, by a whole warp.
__device__ __forceinline__ DistillPart join(const DistillPart* p, int n, float c) {
  const int lane = threadIdx.x & 31;
  DistillPart t = {neg_inf(), neg_inf(), ff(0.f), ff(0.f), ff(0.f), 0};
  if (lane < n) t = p[lane];
  const float mr = warp_max_nan(t.mr), ml = warp_max_nan(t.ml);
  t.rest = t.rest.hi > 0.f ? ff_mul(t.rest, ex2((t.mr - mr) * c)) : ff(0.f);
  t.listed = t.listed.hi > 0.f ? ff_mul(t.listed, ex2((t.ml - ml) * c)) : ff(0.f);
  t.bad = __reduce_or_sync(0xffffffffu, t.bad);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    t.rest = ff_gather(t.rest, shfl_xor(t.rest, o));
    t.listed = ff_gather(t.listed, shfl_xor(t.listed, o));
    t.a = ff_gather(t.a, shfl_xor(t.a, o));
  }
  t.rest = fast_two_sum(t.rest.hi, t.rest.lo);
  t.listed = fast_two_sum(t.listed.hi, t.listed.lo);
  t.mr = mr;
  t.ml = ml;
  return t;
}

// g 2^((z - m) c) of a vector's logits, in their type.
template <int DT>
__device__ __forceinline__ uint4 gradients(const typename Elem<DT>::Vec& v, uint64_t m2, uint64_t c2, uint64_t g2) {
  constexpr int VW = Elem<DT>::VW;
  uint64_t z[VW / 2];
  unpack_pairs<DT>(v, z);
  float x[VW];
#pragma unroll
  for (int k = 0; k < VW / 2; ++k) {
    float a, b;
    f2_split(f2_mul(f2_add(z[k], m2), c2), a, b);
    f2_split(f2_mul(f2(ex2(a), ex2(b)), g2), x[2 * k], x[2 * k + 1]);
  }
  return pack_vec<DT>(x);
}

// Bytes of a CTA's work space behind the held vectors: a bit per logit of the
// slice (the listed ids) and five words per teacher entry.
__host__ __device__ constexpr size_t distill_bytes(int svec, int vw, int K) {
  return (static_cast<size_t>(svec) * vw / 8 + 19) / 16 * 16 + static_cast<size_t>(K) * 20;
}

// The bits of vector v of the slice, a bit per logit.
template <int DT>
__device__ __forceinline__ unsigned vector_bits(const unsigned char* bits, int v) {
  if (DT == 0) return bits[v];
  return (bits[v >> 1] >> ((v & 1) * 4)) & 15u;
}

// Loss, statistics and (grad given) the gradient of the rows: a cluster per
// row.  One pass for the maximum and the sum of the logits that are not listed
// (each thread's sum relative to its own running maximum, joined at the end),
// one for the gradient.  1024 x 128256 bf16, K = 64, with the gradient 134 us (525
// MB, 3.9 TB/s): 69 % of issue slots, and a third of the second read comes from
// HBM again; 1024 x 152064 fp32, K = 256, loss alone 124 us (623 MB, 5.0 TB/s).
template <int DT>
__global__ void __launch_bounds__(kRowThreads, 2) distill_kernel(const __grid_constant__ DistillParams P) {
  using E = Elem<DT>;
  using Vec = typename E::Vec;
  constexpr int VW = E::VW;
  extern __shared__ __align__(128) char smem[];
  __shared__ uint64_t bars[kRowWarps * kMaxRing];
  __shared__ float tred[kRowWarps];
  __shared__ uint64_t ured[kRowWarps];
  __shared__ DistillPart wpart[kRowWarps], part[kMaxCluster];
  __shared__ float2 origin;
  __shared__ int again, late;
  __shared__ float row_max, row_ref, row_alpha, row_beta;
  __shared__ int row_dead;
  const int C = P.sp.C, K = P.K, V = P.sp.V;
  const int rank = cluster_rank();
  const int64_t row = blockIdx.x / C;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  cluster_arrive();  // waited for before the first remote write
  const char* zrow = reinterpret_cast<const char*>(P.z) + row * P.rs * E::ES;
  char* grow = reinterpret_cast<char*>(P.grad) + row * P.grs * E::ES;
  RowSlice<DT, true, false> sl;
  sl.init(smem, bars, P.sp, zrow, rank, warp);
  const float wt = P.weight ? P.weight[row] : 1.f;
  const bool skip = wt == 0.f;
  if (threadIdx.x == 0) again = late = 0;
  const int words = (P.sp.svec * VW + 31) / 32;
  unsigned* bits = reinterpret_cast<unsigned*>(smem + row_bytes(P.sp.rvec, P.sp.stages));
  int32_t* ids = reinterpret_cast<int32_t*>(smem + row_bytes(P.sp.rvec, P.sp.stages) +
                                            distill_bytes(P.sp.svec, VW, 0));
  float* tl = reinterpret_cast<float*>(ids + K);
  float* pj = tl + K;
  float* zj = pj + K;
  float* sj = zj + K;  // p of the entry's id, or -1: not its first entry
  const float ih = P.ih, c = P.c;
  const int lo = sl.base, hi = min(V, lo + P.sp.svec * VW);  // the slice's indices
  Teacher te = {};
  te.pscale = 1.f;
  int bad = 0;
  RunningSum rs;  // over the logits that are not listed
  float zmax = neg_inf();
  if (!skip) {
    sl.load(P.stall[0] == row + 1 && rank == 0 && warp == 0);
    for (int i = threadIdx.x; i < words; i += kRowThreads) bits[i] = 0;
    te = load_teacher<true>(P, row, ids, tl, pj, tred, ured);  // (a barrier: no bits, too)
    bad = te.bad;
    // The loss is sum p (log p - log q), of terms relative to an entry's (the first
    // there is, in a sorted list the largest): logits of student and teacher may lie
    // anywhere, thousands of T apart.
    if (threadIdx.x == kRowThreads - 1) {
      int j = 0;
      while (j < K && ids[j] < 0) ++j;
      const float t0 = j < K ? tl[j] : 0.f, z0 = j < K ? E::scalar(zrow, ids[j]) : 0.f;
      origin = isfinite(t0) && isfinite(z0) ? make_float2(t0, z0) : make_float2(0.f, 0.f);
    }
    // The listed ids of this slice: their logits, and a bit for each.
    for (int j = threadIdx.x; j < K; j += kRowThreads) {
      const int id = ids[j];
      if (id < lo || id >= hi) continue;
      const float z = E::scalar(zrow, id), p = pj[j] * te.pscale;
      const unsigned bit = 1u << ((id - lo) & 31);
      if (atomicOr(&bits[(id - lo) >> 5], bit) & bit) again = 1;
      zj[j] = z;
      sj[j] = p;
      zmax = max_nan(zmax, z);
    }
    __syncthreads();
    if (again) {  // rare: an id listed twice; its first entry stands for them
      for (int j = warp; j < K; j += kRowWarps) {
        const int id = ids[j];
        if (id < lo || id >= hi) continue;
        bool first;
        const float ps = same_id(ids, pj, K, j, lane, first) * te.pscale;
        if (lane == 0) sj[j] = first ? ps : -1.f;
      }
      __syncthreads();
    }
    // the logits that are not listed
    const unsigned char* byte = reinterpret_cast<const unsigned char*>(bits);
    sl.ready();
    sl.groups([&](const Vec(&y)[2], int j) {
      uint64_t z[VW];
      float top = rs.run;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const unsigned listed = j + 32 * u < sl.nv ? vector_bits<DT>(byte, sl.v0 + j + 32 * u) : 0u;
        float x[VW];
        E::unpack(y[u], x);
        if (listed) {
#pragma unroll
          for (int k = 0; k < VW; ++k) {
            x[k] = (listed >> k) & 1u ? neg_inf() : x[k];
            top = max_nan(top, x[k]);
          }
        } else {
          top = vec_max<DT>(y[u], top);
        }
#pragma unroll
        for (int k = 0; k < VW / 2; ++k) z[u * (VW / 2) + k] = f2(x[2 * k], x[2 * k + 1]);
      }
      rs.add(z, top, c);
    });
    if (sl.late) bad |= kTimeout;
    if (P.grad && sl.stages > 0) sl.prime(P.stall[1] == row + 1 && rank == 0 && warp == 0);  // (the second pass's first copies)
  }
  // Each warp's sums, relative to its own maxima.  The rest keeps one of its
  // own: a student may put e^-100 and less of its mass outside the list.
  const float mr = warp_max_nan(rs.run), ml = warp_max_nan(zmax);
  float listed = 0.f, a = 0.f;
  if (!skip) {
    const float mref = ml > neg_inf() ? ml : 0.f;
    for (int j = threadIdx.x; j < K; j += kRowThreads) {
      if (ids[j] < lo || ids[j] >= hi) continue;
      const float p = pj[j] * te.pscale, z = zj[j];
      if (sj[j] >= 0.f) listed += ex2((z - mref) * c);
      const float lead = ((tl[j] - origin.x) - (z - origin.y)) * ih;
      if (p > 0.f && lead < pos_inf()) a += p * lead;
      else if (p > 0.f) bad |= kRuledOut;
    }
  }
  listed = warp_sum_f(listed);
  const float rest = warp_sum_f(rs.at(mr, c));
  a = warp_sum_f(a);
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (lane == 0) {
    DistillPart mine = {mr, ml, ff(rest), ff(listed), ff(a), bad};
    wpart[warp] = mine;
  }
  __syncthreads();
  cluster_wait();
  DistillPart all;
  if (warp == 0) {
    all = join(wpart, kRowWarps, c);
    if (C > 1 && lane < C) *peer(part + rank, lane) = all;
  }
  if (C > 1) {
    cluster_sync();
    if (warp == 0) all = join(part, C, c);
  }
  // The row's scalars, by a warp (a lane each for what takes longest).
  FF gap, total;  // log of the rest's largest weight; the row's sum
  float r = 0.f;
  bool dead = false, has_rest = false;
  if (warp == 0) {
    const float ur = all.mr, mx = max_nan(all.mr, all.ml);
    dead = skip || (all.bad & ~kRuledOut) || !(mx > neg_inf() && mx < pos_inf());
    gap = over(ur, mx, ih, P.il);
    auto times = [](FF x, FF y) { return ff_gather(ff_times(x, y.hi), ff(x.hi * y.lo)); };
    const FF e = exp_pair(lane == 0 ? gap : over(all.ml, mx, ih, P.il));
    const FF far = shfl(e, 0), near = shfl(e, 1);
    // all.rest is relative to ur, `total` to mx
    const FF listed_sum = all.listed.hi > 0.f ? times(all.listed, near) : ff(0.f);
    total = ff_gather(listed_sum, all.rest.hi > 0.f ? times(all.rest, far) : ff(0.f));
    total = fast_two_sum(total.hi, total.lo);
    const float recip = 1.f / (lane == 0 ? total.hi : all.rest.hi);
    const float inv = __shfl_sync(0xffffffffu, recip, 0), inv_rest = __shfl_sync(0xffffffffu, recip, 1);
    const float m = te.total(P.tlse != nullptr).hi;
    if (P.tail) r = static_cast<float>((1ll << 40) - static_cast<int64_t>(te.mass)) * (1.f / kFixed);
    if (r < kNoTail) r = 0.f;
    // alpha q_v = m q_v - r s share_v, share_v = exp((z_v - ur) / T) / all.rest.
    // (A rest of the type's lowest values below others is masked: no mass.)
    float beta = m, ref = mx, alpha = m * inv;
    has_rest = all.rest.hi > 0.f && (far.hi > 0.f || ur > E::lowest());
    if (r > 0.f && has_rest) {
      beta = m + r;  // (alpha + r / (1 - s), whose two large terms cancel)
      ref = ur;
      alpha = m * (far.hi * inv) - r * (listed_sum.hi * inv) * inv_rest;
    }
    beta *= inv;
    if (lane == 0) {
      row_dead = dead;
      row_max = mx;
      row_ref = ref;
      row_alpha = alpha;
      row_beta = beta;
      if (rank == 0) {
        if (P.stats)
          P.stats[row] = dead ? make_float4(__int_as_float(0x7fc00000), 0.f, 0.f, 0.f) : make_float4(ref, alpha, mx, beta);
        if (P.status) P.status[row] = skip || !dead ? 0 : (all.bad & ~kRuledOut) | (mx > neg_inf() && mx < pos_inf() ? 0 : kNonFinite);
      }
    }
  }
  if (P.grad) __syncthreads();
  if (warp == 0 && rank == 0) {  // the loss, while the others start on the gradient
    FF l = log_pair(lane == 0 ? total.hi : lane == 1 ? all.rest.hi : lane == 2 ? r : te.sum());
    if (lane < 2) l.lo += lane == 0 ? __fdividef(total.lo, total.hi) : __fdividef(all.rest.lo, all.rest.hi);
    const FF lt = shfl(l, 0), lrest = shfl(l, 1), lr = shfl(l, 2), ln = P.tlse ? ff(te.L) : shfl(l, 3);
    FF loss = ff(0.f);
    if (te.mass) {  // log p - log q at the origin, times m
      const FF g = over(max_nan(all.mr, all.ml), origin.y, ih, P.il), o = over(origin.x, P.tlse ? 0.f : te.tmax, ih, P.il);
      const FF d = ff_gather(ff_gather(g, lt), ff_gather(o, ff_neg(ln))), m = te.total(P.tlse != nullptr);
      loss = ff_gather(all.a, ff_gather(ff_times(d, m.hi), ff(d.hi * m.lo)));
    }
    if (r > 0.f && has_rest)
      loss = ff_gather(loss, ff_times(ff_gather(ff_gather(lt, ff_neg(gap)), ff_gather(lr, ff_neg(lrest))), r));
    const bool infinite = (all.bad & kRuledOut) || (r > 0.f && !has_rest);
    if (lane == 0) P.loss[row] = dead ? 0.f : wt * (infinite ? pos_inf() : loss.hi + loss.lo);
  }
  if (!P.grad) return;
  dead = row_dead;
  const float mx = row_max, ref = row_ref;
  const float f = wt * ih;
  const float ga = f * row_alpha;
  const uint64_t c2 = f2(c, c), m2 = f2(-ref, -ref), g2 = f2(ga, ga);
  if (skip) {  // (nothing was copied)
    for (int j0 = 0; j0 < sl.nv; j0 += 32)
      store_warp<DT>(grow, sl.index(j0 + lane), V, j0 + lane < sl.nv, make_uint4(0u, 0u, 0u, 0u));
    return;
  }
  sl.groups([&](const Vec(&y)[2], int j) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint4 w = dead ? make_uint4(0u, 0u, 0u, 0u) : gradients<DT>(y[u], m2, c2, g2);
      store_warp<DT>(grow, sl.index(j + 32 * u), V, j + 32 * u < sl.nv, w);
    }
  });
  if (dead) return;
  if (sl.late) {
    for (int r = 0; r < C; ++r) *peer(&late, r) = 1;
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
  }
  // (Without release: it would wait for this pass's stores, 3 % of the call.)
  if (sl.stages > 0 && C > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  __syncthreads();  // the listed ids' gradients go over what was just written
  const float b = row_beta;
  const FF lb = log_pair(b), ln = te.norm(P.tlse != nullptr);
  for (int j = threadIdx.x; j < K; j += kRowThreads) {
    const int id = ids[j];
    if (id < lo || id >= hi || sj[j] < 0.f) continue;
    store_elem<DT>(grow, id, f * listed_grad(P, te, zj[j], tl[j], pj[j] * te.pscale, sj[j], mx, b, lb, ln));
  }
  // A copy of this pass that was late, in any CTA: the row has no result.
  if (sl.stages > 0 && C > 1) cluster_wait();
  if (!late) return;
  __syncthreads();
  for (int j0 = 0; j0 < sl.nv; j0 += 32)
    store_warp<DT>(grow, sl.index(j0 + lane), V, j0 + lane < sl.nv, make_uint4(0u, 0u, 0u, 0u));
  if (rank == 0 && threadIdx.x == 0) {
    P.loss[row] = 0.f;
    if (P.stats) P.stats[row] = make_float4(__int_as_float(0x7fc00000), 0.f, 0.f, 0.f);
    if (P.status) P.status[row] = kTimeout;
  }
}

// The gradient from the statistics of an earlier distill_kernel: one pass, a
// CTA per piece of a row, of kBackGroups groups of kBackVecs vectors a thread (the
// next group's loads ahead of this one's stores).  Bound by HBM: 1024 x 152064
// fp32 214 us (1246 MB, 5.8 TB/s).
constexpr int kBackVecs = 4, kBackGroups = 4;
__host__ __device__ constexpr int back_piece(int vw) { return kRowThreads * kBackVecs * kBackGroups * vw; }

template <int DT>
__global__ void __launch_bounds__(kRowThreads, 2) distill_backward_kernel(const __grid_constant__ DistillParams P,
                                                                          int pieces) {
  using E = Elem<DT>;
  using Vec = typename E::Vec;
  constexpr int VW = E::VW;
  extern __shared__ __align__(128) char smem[];
  __shared__ float tred[kRowWarps];
  __shared__ uint64_t ured[kRowWarps];
  __shared__ Teacher te;
  const int64_t row = blockIdx.x / pieces;
  const int piece = blockIdx.x % pieces;
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
  const bool dead = wt == 0.f || st.x != st.x;
  const float c = P.c;
  const float f = dead ? 0.f : wt * up * P.ih;
  const float ga = f * st.y;
  // vectors at 16-byte boundaries of memory: `off` places before the row's first logit
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(zrow) & 15) / E::ES;
  constexpr int per = kRowThreads * kBackVecs * VW;
  const int i0 = piece * per * kBackGroups - off, i1 = min(V, i0 + per * kBackGroups);
  const uint64_t c2 = f2(c, c), m2 = f2(-st.x, -st.x), g2 = f2(ga, ga);
  auto load = [&](int at, Vec(&v)[kBackVecs]) {
#pragma unroll
    for (int k = 0; k < kBackVecs; ++k) {
      const int i = at + (k * kRowThreads + static_cast<int>(threadIdx.x)) * VW;
      if (dead || i >= i1) continue;
      if (i >= 0 && i + VW <= V) {
        v[k] = E::vec(zrow, i);
      } else {
        typename E::Raw* d = reinterpret_cast<typename E::Raw*>(&v[k]);
#pragma unroll
        for (int e = 0; e < VW; ++e) d[e] = (i + e >= 0 && i + e < V) ? E::raw(zrow, i + e) : E::neg_inf_raw();
      }
    }
  };
  Vec v[kBackVecs];
  load(i0, v);
  if (!dead) {  // the teacher's entries, while the first loads run
    const Teacher t = load_teacher<false>(P, row, ids, tl, pj, tred, ured);
    if (threadIdx.x == 0) te = t;
  }
#pragma unroll 1
  for (int at = i0; at < i1; at += per) {
    Vec now[kBackVecs];
#pragma unroll
    for (int k = 0; k < kBackVecs; ++k) now[k] = v[k];
    if (at + per < i1) load(at + per, v);  // (ahead of this group's stores)
#pragma unroll
    for (int k = 0; k < kBackVecs; ++k) {
      const int i = at + (k * kRowThreads + static_cast<int>(threadIdx.x)) * VW;
      if (at + (k * kRowThreads + warp * 32) * VW >= i1) break;  // (the same for the whole warp)
      const bool on = i < i1;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (on && !dead) w = gradients<DT>(now[k], m2, c2, g2);
      store_warp<DT>(grow, i, V, on, w);
    }
  }
  if (dead) return;
  __syncthreads();  // the listed ids' gradients go over what was just written
  const FF lb = log_pair(st.w), ln = te.norm(P.tlse != nullptr);
  // Each warp gathers its entries of this piece, then takes them a lane each.
  int own = -1, held = 0;
  float own_ps = 0.f;
  auto store = [&] {
    if (own >= 0)
      store_elem<DT>(grow, ids[own], f * listed_grad(P, te, E::scalar(zrow, ids[own]), tl[own], pj[own] * te.pscale,
                                                     own_ps, st.z, st.w, lb, ln));
    own = -1;
    held = 0;
  };
  for (int j = warp; j < K; j += kRowWarps) {
    const int id = ids[j];
    if (id < max(i0, 0) || id >= i1) continue;  // (i0 lies before a row that starts inside a vector; absent: -1)
    bool first;
    const float ps = same_id(ids, pj, K, j, lane, first) * te.pscale;
    if (!first) continue;
    if (lane == held) {
      own = j;
      own_ps = ps;
    }
    if (++held == 32) store();
  }
  store();
}

}  // namespace specv
