// Sampling with temperature, top-k, top-p and min-p, and the k largest logits.
//
// A row's kept set is a prefix of its tokens in the order (logit descending,
// index ascending), so it is named by one logit and one index: kept iff
// z > zc, or z == zc and index <= ic.  The cut is found by a histogram of
// y = z log2(e) / T in bins of 1/64 below the maximum (counts for top-k, masses
// for top-p), which names the few bins that the cut can lie in; their tokens
// are gathered, sorted and summed exactly.  A band too full to gather is split
// by the bits of the logits, then (all equal) by index.
//
// Whole numbers come out of the sums of weights 2^(y - max) (the cut, the
// token), and a sum in plain fp32 moves the cut of a flat distribution in one
// row of a hundred.  So a weight is held to about 2^-31 of it, in two forms:
//   for the cut: 2^(-d/64) (v 2^-bits + e), d its bin, v a whole number (the
//     bins sum v exactly), e the rest in fp32;
//   for the draw: h + l, h = 2^(-d/64) rounded to fp32, l the rest (their sums
//     recover each rounding).
// Totals are 64-bit integers in units of 2^-fbits of the largest weight (an SM
// does two fp64 operations a clock: a block's reductions in fp64 cost more than
// its passes over the row).
#pragma once

#include "distill_kernel.cuh"  // block_max_nan

namespace specv {

constexpr int kGrid = 64;                 // bins per unit of log2
constexpr int kWindow = 48;               // units below the maximum that carry weight
constexpr int kBins = kGrid * kWindow + 16;
constexpr int kLocal = 2048;              // tokens of a band that a CTA collects
constexpr int kCap = 1024;                // ... and that rank 0 works on
constexpr int kBadFilter = 64;
constexpr float kMagic = 196608.f;        // 1.5 * 2^17: adding it rounds to 1/64
// kSlack: sums equal within 2^-36 (x >> 36) count as equal, so that equal
// weights which meet a border exactly fall on its right side.

struct BinTable {
  uint64_t e[kGrid];  // 2^(63 + j/64)
  float2 p[kGrid];    // 2^(j/64): rounded to fp32, and what that leaves of it
};

struct FilterParams {
  RowSplit sp;
  int32_t rows, R;        // rows; rows per parameter entry
  const void* z;
  int64_t bs, rs;         // strides of batch entries and of the R rows in one
  const float* temp;
  const int32_t* top_k;   // or NULL, as the next two
  const float* top_p;
  const float* min_p;
  const float* u;         // or NULL: no token
  int32_t* tokens;
  float* prob;
  int32_t* kept;
  void* out;              // filtered logits, or NULL
  int64_t obs, ors;
  int32_t* status;
  BinTable tab;
};

struct TopParams {
  RowSplit sp;
  int32_t rows, k;
  const void* z;
  int64_t rs;
  double invT;   // 1 / T
  float c;       // log2(e) / T
  int32_t* ids;
  float* values;
  float* lse;
  int32_t* status;
};

// fp32 bits in an unsigned order; -0 and +0 get the same key.
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);
  return b ^ ((b & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number

// The row's exponent scale: y = (z - shift) (chi + clo), gm = the maximum's
// place on the grid of 1/64.  Weights are relative to 2^(gm / 64).
struct Scale {
  float shift, chi, clo, gmf;  // gmf = gm / 64
  int gm;

  // c = log2(e) / T.  bf16: chi has 16 digits, so that its products are exact.
  template <int DT>
  __device__ void set_factor(double c) {
    chi = static_cast<float>(c);
    if (DT == 0) chi = __int_as_float(__float_as_int(chi) & 0xffffff00);
    clo = static_cast<float>(c - static_cast<double>(chi));
  }
  __device__ void set_max(float m) {
    // |y| stays within the rounding trick's range; shifted logits are exact
    // where they carry weight (within 48 units of a maximum of 2^14 units).
    shift = fabsf(m) * chi > 16384.f ? m : 0.f;
    const float r = __fadd_rn(__fmul_rn(m - shift, chi), kMagic);
    gm = __float_as_int(r) - __float_as_int(kMagic);
    gmf = __fadd_rn(r, -kMagic);
  }
  // Distance from the maximum in bins: rounding is monotone, so 0 <= bin <=
  // 48 * 64 + 3 for a logit of the window.  CLAMP: for any logit below the
  // maximum.
  template <bool CLAMP>
  __device__ __forceinline__ int bin(float z) const {
    float p = __fmul_rn(z - shift, chi);
    if (CLAMP) p = fmaxf(p, -60000.f);
    const float r = __fadd_rn(p, kMagic);
    const int d = gm + __float_as_int(kMagic) - __float_as_int(r);
    return CLAMP ? min(d, kBins - 1) : d;
  }
  // What y leaves beside its bin (|g| <= 2^-7) and the bin's place below the
  // maximum.
  template <int DT>
  __device__ __forceinline__ float split(float z, int& d, float& cb) const {
    const float x = z - shift;
    const float p = __fmul_rn(x, chi);
    const float r = __fadd_rn(p, kMagic);
    cb = __fadd_rn(r, -kMagic);
    d = gm + __float_as_int(kMagic) - __float_as_int(r);
    const float g = __fadd_rn(p, -cb);  // exact
    return DT == 0 ? fmaf(x, clo, g) : g + fmaf(x, clo, fmaf(x, chi, -p));
  }
  // h and l of a logit of the window, d its bin.
  template <int DT>
  __device__ __forceinline__ void pair(float z, const float2* tab, float& h, float& l, int& d) const {
    float cb;
    const float g = split<DT>(z, d, cb);
    const float2 t = tab[(-d) & (kGrid - 1)];
    h = __int_as_float(__float_as_int(t.x) - (((d + kGrid - 1) & -kGrid) << 17));
    // 2^g - 1 to 2^-34
    l = h * fmaf(g, fmaf(g, fmaf(g, 0.05550411f, 0.24022651f), 0.69314718f), t.y);
  }
  // d, v and e 2^(-d/64) of a logit of the window; lin = ln 2 * 2^bits, inv =
  // 2^-bits, one = 2^bits less kRound's bits.
  template <int DT>
  __device__ __forceinline__ void weight(float z, float lin, float inv, int one, int& d, uint32_t& v, float& e) const {
    float cb;
    const float g = split<DT>(z, d, cb);
    const float n = __fadd_rn(__fmul_rn(g, lin), kRound);
    v = static_cast<uint32_t>(__float_as_int(n) + one);
    // 2^g - 1 for |g| <= 2^-7 (the next term is below 2^-34)
    const float t = __fmul_rn(g, fmaf(g, fmaf(g, 0.05550411f, 0.24022651f), 0.69314718f));
    e = __fmul_rn(ex2(cb - gmf), fmaf(__fadd_rn(n, -kRound), -inv, t));
  }
};

// A running sum of weights h + l.  Both sums stay above any addend (a weight is
// below 1.02; its l is below 2^-7 in size, and a thread adds a few hundred), so
// each rounding's error is recovered exactly and kept in c: equal weights sum
// to their exact multiple to about 2^-38.
struct PairSum {
  float a = 4.f, b = 4.f, c = 0.f;
  __device__ __forceinline__ void add(float h, float l) {
    const float s = __fadd_rn(a, h), t = __fadd_rn(b, l);
    c += __fadd_rn(h, -__fadd_rn(s, -a));
    c += __fadd_rn(l, -__fadd_rn(t, -b));
    a = s;
    b = t;
  }
  __device__ __forceinline__ uint64_t fixed(float unit) const {  // unit = 2^fbits
    return static_cast<uint64_t>(__float2ll_rn((a - 4.f) * unit) + __float2ll_rn((b - 4.f) * unit) +
                                 __float2ll_rn(c * unit));
  }
};

__device__ __forceinline__ uint64_t warp_sum_u(uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// What the CTA of rank 0 decides and every CTA reads.
struct Decision {
  float zc;
  int32_t ic;
  int32_t count;      // tokens in the band gathered last
  uint32_t kmin, kmax;
  int32_t tie_seg, tie_rank;
  int32_t seg;        // the segment the token lies in
  uint64_t rem;       // u W minus what lies before that segment
  uint64_t W;
  int32_t kept;
  int32_t fallback;
};

struct FilterShared {
  uint64_t bars[kRowWarps];
  BinTable tab;
  uint32_t hist[kLocal * 2]; // the CTA's histogram; then the band's keys (8 bytes each) that it collects
  uint32_t total[kBins];     // the row's histogram; then the warps' queues; then, in rank 0, the band's keys
  float xmax[kMaxCluster];
  uint64_t xsum[kMaxCluster];
  float xexp[kMaxCluster];
  int32_t xbad[kMaxCluster];
  int32_t xidx[kMaxCluster];
  int32_t xcount[kMaxCluster];
  uint64_t scratch[kRowWarps];
  float fscratch[kRowWarps];
  int32_t iscratch[kRowWarps];
  // rank 0: per segment of the row
  uint64_t segsum[kMaxSegs];
  int32_t segabove[kMaxSegs], segband[kMaxSegs];
  uint32_t segkmin[kMaxSegs], segkmax[kMaxSegs];
  int32_t ngather;
  int32_t lo, hi;
  int32_t before;
  int32_t above;
  Scale sc;
  float zf, zt;
  Decision dec;
};
static_assert(kBins <= kLocal * 2 && kCap * 2 <= kBins && kRowWarps * 128 <= kBins, "arrays that share memory fit");

// The set being cut and the band of it that is looked at: tokens above the
// band are certainly kept by the cut, those below certainly not.
struct Band {
  bool by_key;
  int lo, hi;            // bins
  float edge;            // every token of the band is >= edge
  uint32_t kmin, kmax;   // keys
};

template <int DT, bool CLAMP>
struct FilterRow {
  FilterShared& S;
  RowSlice<DT> sl;
  Scale sc;
  int rank, C, V, lane, warp;
  float zc;
  int ic;
  int fbits;    // sums are in units of 2^-fbits, so that V weights stay below 2^62
  int bits;     // a bin's v in units of 2^-bits, so that V of them fit 32 bits
  int one;      // for Scale::weight, as the next two
  float lin, inv;
  float unit;   // 2^fbits

  __device__ void set_units() {
    const int n = 32 - __clz(V);
    fbits = min(44, 62 - n);
    bits = min(14, 31 - n);
    unit = __int_as_float((127 + fbits) << 23);
    inv = __int_as_float((127 - bits) << 23);
    lin = 0.69314718f * __int_as_float((127 + bits) << 23);
    one = (1 << bits) - __float_as_int(kRound);
  }

  __device__ FilterRow(FilterShared& s) : S(s) {}

  __device__ __forceinline__ bool in_set(float z, int i) const { return z > zc || (z == zc && i <= ic); }

  // 0: above the band, 1: in it, 2: below
  __device__ __forceinline__ int place(float z, const Band& b) const {
    if (b.by_key) {
      const uint32_t k = order_key(z);
      return k > b.kmax ? 0 : k >= b.kmin ? 1 : 2;
    }
    const int d = sc.template bin<CLAMP>(z);
    return d < b.lo ? 0 : d <= b.hi ? 1 : 2;
  }

  // The row's histogram into S.total on every CTA.  Barriers: the cluster's,
  // twice.  Before it: S.hist filled by this CTA (and a __syncthreads).
  __device__ void merge(int bins) {
    cluster_sync();
    const int per = (bins / 4 + C - 1) / C;
    const int b0 = rank * per, b1 = min(bins / 4, b0 + per);
    for (int b = b0 + static_cast<int>(threadIdx.x); b < b1; b += kRowThreads) {
      uint4 t = make_uint4(0u, 0u, 0u, 0u);
      for (int r0 = 0; r0 < C; r0 += 8) {  // loads of eight CTAs in flight
        uint4 x[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          x[q] = r0 + q < C ? reinterpret_cast<const uint4*>(peer(S.hist, r0 + q))[b] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          t.x += x[q].x;
          t.y += x[q].y;
          t.z += x[q].z;
          t.w += x[q].w;
        }
      }
      for (int r = 0; r < C; ++r) reinterpret_cast<uint4*>(peer(S.total, r))[b] = t;
    }
    cluster_sync();
  }

  // Exclusive prefix over the block's threads; `all` gets the total.
  template <typename T>
  __device__ T block_scan(T x, T* scratch, T& all) {
    T inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    T base = 0;
    all = 0;
    for (int w = 0; w < kRowWarps; ++w) {
      if (w < warp) base += scratch[w];
      all += scratch[w];
    }
    return base + inc - x;
  }

  __device__ void clear_hist(int bins) {
    for (int b = threadIdx.x; b < bins / 4; b += kRowThreads) reinterpret_cast<uint4*>(S.hist)[b] = make_uint4(0u, 0u, 0u, 0u);
    if (threadIdx.x == 0) {
      S.ngather = 0;
      S.lo = S.hi = INT_MAX;
    }
    __syncthreads();
  }

  // Collects the band's tokens, a list in each CTA, and leaves at rank 0, per
  // segment, the number and (sums) the weight of the tokens above the band,
  // and the band's count and range of keys.  Ends with a cluster barrier.
  // Where a warp's vectors hold few of these tokens (peaked rows), it queues
  // them and works on 32 at a time; where they hold many, it works in place.
  __device__ void gather(const Band& b, bool sums) {
    PairSum acc;
    int above = 0, band = 0;
    uint32_t kmin = 0xffffffffu, kmax = 0;
    uint64_t* list = reinterpret_cast<uint64_t*>(S.hist);
    uint2* queue = reinterpret_cast<uint2*>(S.total) + warp * 64;
    const float edge = b.edge;
    auto work = [&](bool cand, float z, int i) {
      const int pl = place(z, b);
      const bool over = cand && pl == 0;
      above += over;
      if (!CLAMP && sums) {
        float h, l;
        int d;
        sc.template pair<DT>(z, S.tab.p, h, l, d);
        acc.add(over ? h : 0.f, over ? l : 0.f);
      }
      if (cand && pl == 1) {
        ++band;
        const uint32_t key = order_key(z);
        kmin = min(kmin, key);
        kmax = max(kmax, key);
        const int pos = atomicAdd(&S.ngather, 1);
        if (pos < kLocal) list[pos] = (static_cast<uint64_t>(~key) << 32) | static_cast<uint32_t>(i);
      }
    };
    int queued = 0;
    auto flush = [&](int n) {
      __syncwarp();
      const uint2 it = queue[lane];
      work(lane < n, lane < n ? __uint_as_float(it.x) : edge_safe(), it.y);
    };
    for (int j0 = 0; j0 < sl.nv; j0 += 32) {
      const int j = j0 + lane;
      float z[Elem<DT>::VW];
      float top = neg_inf();
      if (j < sl.nv) {
        Elem<DT>::unpack(sl.data[sl.v0 + j], z);
#pragma unroll
        for (int k = 0; k < Elem<DT>::VW; k += 2) top = max3(top, z[k], z[k + 1]);
      }
      const unsigned lanes = __ballot_sync(0xffffffffu, top >= edge);
      if (!lanes) continue;
      const int i0 = sl.base + (sl.v0 + j) * Elem<DT>::VW;
      if (__popc(lanes) >= 24) {  // most lanes hold one at least
#pragma unroll
        for (int k = 0; k < Elem<DT>::VW; ++k) {
          const bool cand = top >= edge && z[k] >= edge && in_set(z[k], i0 + k);
          work(cand, cand ? z[k] : edge_safe(), i0 + k);
        }
        continue;
      }
#pragma unroll
      for (int k = 0; k < Elem<DT>::VW; ++k) {
        const bool cand = top >= edge && z[k] >= edge && in_set(z[k], i0 + k);
        const unsigned mask = __ballot_sync(0xffffffffu, cand);
        if (cand) queue[queued + __popc(mask & ((1u << lane) - 1))] = make_uint2(__float_as_uint(z[k]), i0 + k);
        queued += __popc(mask);
        if (queued >= 32) {
          flush(32);
          queued -= 32;
          const uint2 rest = queue[32 + lane];
          __syncwarp();
          if (lane < queued) queue[lane] = rest;
          __syncwarp();
        }
      }
    }
    if (queued > 0) flush(queued);
    const uint64_t w = warp_sum_u(acc.fixed(unit));
    above = __reduce_add_sync(0xffffffffu, above);
    band = __reduce_add_sync(0xffffffffu, band);
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    if (lane == 0) {
      const int s = rank * kRowWarps + warp;
      peer(S.segsum, 0)[s] = w;
      peer(S.segabove, 0)[s] = above;
      peer(S.segband, 0)[s] = band;
      peer(S.segkmin, 0)[s] = kmin;
      peer(S.segkmax, 0)[s] = kmax;
    }
    __syncthreads();
    push_all(S.xcount, rank, C, S.ngather);
    cluster_sync();
  }

  // Tokens in the band gathered last (more than kCap: not all were collected).
  __device__ int gathered() const {
    int n = 0;
    bool over = false;
    for (int r = 0; r < C; ++r) {
      over |= S.xcount[r] > kLocal;
      n += S.xcount[r];
    }
    return over ? max(n, kCap + 1) : n;
  }

  // Rank 0: the n <= kCap collected keys into S.total (ends with a barrier).
  __device__ void pull(int n) {
    uint64_t* list = reinterpret_cast<uint64_t*>(S.total);
    for (int t = threadIdx.x; t < n; t += kRowThreads) {
      int r = 0, i = t;
      while (i >= S.xcount[r]) i -= S.xcount[r++];
      list[t] = reinterpret_cast<const uint64_t*>(peer(S.hist, r))[i];
    }
    __syncthreads();
  }

  // Sorts n <= kCap keys ascending: logit descending, index ascending.
  __device__ void sort(uint64_t* list, int n) {
    int P = 16;
    while (P < n) P <<= 1;
    if (P <= kRowThreads / 2) {  // few: G threads count the keys before each
      const int G = kRowThreads / P, i = threadIdx.x / G, sub = threadIdx.x % G;
      const uint64_t x = i < n ? list[i] : 0;
      int before = 0;
      for (int j = sub; j < n; j += G) before += list[j] < x;
      for (int o = G / 2; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
      __syncthreads();
      if (sub == 0 && i < n) list[before] = x;
      __syncthreads();
      return;
    }
    // two keys a thread (i = 2 t and 2 t + 1), steps below 64 within a warp
    uint64_t a = ~0ull, b = ~0ull;
    const int i = 2 * threadIdx.x;
    if (i < n) a = list[i];
    if (i + 1 < n) b = list[i + 1];
    for (int size = 2; size <= P; size <<= 1) {
      const bool up = (i & size) == 0;
      for (int step = size >> 1; step > 0; step >>= 1) {
        if (step == 1) {
          if ((a > b) == up) {
            const uint64_t t = a;
            a = b;
            b = t;
          }
          continue;
        }
        uint64_t x, y;
        if (step < 64) {
          x = __shfl_xor_sync(0xffffffffu, a, step >> 1);
          y = __shfl_xor_sync(0xffffffffu, b, step >> 1);
        } else {
          __syncthreads();
          if (i < P) {
            list[i] = a;
            list[i + 1] = b;
          }
          __syncthreads();
          x = i < P ? list[i ^ step] : a;
          y = i < P ? list[(i + 1) ^ step] : b;
        }
        const bool lower = (i & step) == 0;
        if ((a > x) == (lower == up)) a = x;
        if ((b > y) == (lower == up)) b = y;
      }
    }
    __syncthreads();
    if (i < n) list[i] = a;
    if (i + 1 < n) list[i + 1] = b;
    __syncthreads();
  }

  // Block-wide sum (every thread gets it).
  __device__ uint64_t block_sum_u(uint64_t x) {
    x = warp_sum_u(x);
    __syncthreads();
    if (lane == 0) S.scratch[warp] = x;
    __syncthreads();
    x = 0;
    for (int w = 0; w < kRowWarps; ++w) x += S.scratch[w];
    return x;
  }

  // Rank 0: totals over the segments of the gather before.
  __device__ void seg_totals(uint64_t& w, int& above, int& band) {
    const int n = C * kRowWarps;
    uint64_t x = 0, y = 0;
    if (static_cast<int>(threadIdx.x) < n) {
      x = S.segsum[threadIdx.x];
      y = (static_cast<uint64_t>(S.segabove[threadIdx.x]) << 32) | static_cast<uint32_t>(S.segband[threadIdx.x]);
    }
    w = block_sum_u(x);
    y = block_sum_u(y);
    above = static_cast<int>(y >> 32);
    band = static_cast<int>(y & 0xffffffffu);
  }

  __device__ void publish() {  // rank 0's decision to every CTA
    __syncthreads();
    if (rank == 0) {
      const Decision d = S.dec;
      if (static_cast<int>(threadIdx.x) < C && threadIdx.x > 0) *peer(&S.dec, static_cast<int>(threadIdx.x)) = d;
    }
    cluster_sync();
  }

  // v 2^-bits 2^(-d/64) in units of 2^-fbits.
  __device__ __forceinline__ uint64_t mass(uint32_t v, int d) const {
    const uint64_t t = S.tab.e[(-d) & (kGrid - 1)];
    const uint64_t x = static_cast<uint64_t>(v) * (t >> 32) + ((static_cast<uint64_t>(v) * (t & 0xffffffffu)) >> 32);
    const int s = bits + 31 - fbits - ((-d) >> 6);  // 0 or 1, and the halvings of d
    return s > 0 ? (x + (1ull << (s - 1))) >> s : x;
  }

  // A token's weight without its e, which is added to `low`.
  __device__ __forceinline__ uint64_t part_weight(float z, float& low) const {
    int d;
    uint32_t v;
    float e;
    sc.template weight<DT>(z, lin, inv, one, d, v, e);
    low += e;
    return mass(v, d);
  }

  // A logit of the window, for lanes without one of their own.
  __device__ __forceinline__ float edge_safe() const { return sc.shift; }

  // A token's weight for the draw.
  __device__ __forceinline__ uint64_t draw_weight(float z) const {
    float h, l;
    int d;
    sc.template pair<DT>(z, S.tab.p, h, l, d);
    return static_cast<uint64_t>(__float2ll_rn(h * unit) + __float2ll_rn(l * unit));
  }

  // A token's weight for the cut.
  __device__ __forceinline__ uint64_t fixed_weight(float z) const {
    float e = 0.f;
    const uint64_t w = part_weight(z, e);
    return w + static_cast<uint64_t>(__float2ll_rn(e * unit));
  }

  // Bins -> the band between the first bin where the cut may lie and the
  // first where it must.  COUNT: the goal-th token; else the mass `share` of
  // the whole set's, left in goal (the bins' masses are good to 2^-bits; the
  // rest of each weight, summed, is in S.xsum).  S.before: the count before the
  // band.  False if the set ends before the goal-th token.
  template <bool COUNT>
  __device__ bool find_bins(uint64_t& goal, float share, Band& b) {
    // warp w holds bins [w * kBinsPerWarp, ...), a lane every 32nd
    constexpr int kBinsPerWarp = (kBins + kRowWarps - 1) / kRowWarps, per = (kBinsPerWarp + 31) / 32;
    const int b0 = warp * kBinsPerWarp, b1 = min(kBins, b0 + kBinsPerWarp);
    uint64_t v[per], x = 0;
#pragma unroll
    for (int q = 0; q < per; ++q) {
      const int d = b0 + q * 32 + lane;
      const uint32_t n = d < b1 ? S.total[d] : 0u;
      v[q] = COUNT ? n : n ? mass(n, d) : 0;
      x += v[q];
    }
    x = warp_sum_u(x);
    if (lane == 0) S.scratch[warp] = x;
    __syncthreads();
    uint64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) {
      if (w < warp) before += S.scratch[w];
      all += S.scratch[w];
    }
    if (COUNT) {
      if (all < goal) return false;
    } else {
      for (int r = 0; r < C; ++r) all += S.xsum[r];
      goal = __umul64hi(all, __float2ull_rd(share * 18446744073709551616.f)) + 1;
      goal -= goal >> 36;  // kSlack
    }
    const uint64_t end = before + x;
    if (x && end + (COUNT ? 0 : (end >> bits) + 1) >= goal && (before < goal + (COUNT ? 0 : (goal >> (bits - 1)) + 2))) {
      // the cut may lie among this warp's bins
      uint64_t run = before;
#pragma unroll
      for (int q = 0; q < per; ++q) {
        uint64_t inc = v[q];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        const uint64_t mine = run + inc;
        const uint64_t slack = COUNT ? 0 : (mine >> bits) + 1;
        const int d = b0 + q * 32 + lane;
        const unsigned may = __ballot_sync(0xffffffffu, v[q] && mine + slack >= goal);
        const unsigned must = __ballot_sync(0xffffffffu, v[q] && mine - slack >= goal);
        if (may && lane == __ffs(may) - 1) {
          atomicMin(&S.lo, d);
          if (COUNT && mine - v[q] < goal) S.before = static_cast<int32_t>(mine - v[q]);
        }
        if (must) {
          if (lane == __ffs(must) - 1) atomicMin(&S.hi, d);
          break;
        }
        run = __shfl_sync(0xffffffffu, mine, 31);
      }
    }
    __syncthreads();
    b.by_key = false;
    b.lo = S.lo == INT_MAX ? kBins - 1 : S.lo;
    b.hi = S.hi == INT_MAX ? kBins - 1 : S.hi;
    // 64 y >= gm - hi - 1/2 for every token of the band, with room for rounding
    const float e = sc.shift + (static_cast<float>(sc.gm - b.hi) - 0.5f) / (static_cast<float>(kGrid) * sc.chi);
    b.edge = b.hi >= kBins - 1 ? kNegMax : fmaxf(e - 1e-6f * (fabsf(e) + fabsf(sc.shift)) - 1e-30f, kNegMax);
    return true;
  }

  // Narrows a band too full to gather: counts by key over [kmin, kmax] into
  // 2048 bins.  count: the cut is the goal-th token of the band; else the
  // mass `goal` into it.
  __device__ void narrow(Band& b, bool count, uint64_t goal) {
    const uint32_t kmin = b.kmin, kmax = b.kmax;
    int shift = 0;
    while (((kmax - kmin) >> shift) >= 2048u) ++shift;
    clear_hist(2048);
    sl.each([&](float z, int i) {
      if (z >= b.edge && in_set(z, i) && place(z, b) == 1) {
        const uint32_t key = order_key(z);
        if (key >= kmin && key <= kmax) atomicAdd(&S.hist[(kmax - key) >> shift], 1u);
      }
    });
    __syncthreads();
    merge(2048);
    constexpr int per = 2048 / kRowThreads;
    const int b0 = threadIdx.x * per;
    uint64_t hi_x = 0, lo_x = 0, hw[per], lw[per];
    for (int q = 0; q < per; ++q) {
      const uint32_t n = S.total[b0 + q];
      const uint32_t top = kmax - (static_cast<uint32_t>(b0 + q) << shift);
      const uint32_t span = (1u << shift) - 1;
      const uint32_t low = top - kmin < span ? kmin : top - span;
      hw[q] = n == 0 ? 0 : count ? n : n * (fixed_weight(key_value(top)) + 1);
      lw[q] = n == 0 ? 0 : count ? n : n * fixed_weight(key_value(low));
      hi_x += hw[q];
      lo_x += lw[q];
    }
    uint64_t all;
    uint64_t hi_run = block_scan(hi_x, S.scratch, all);
    uint64_t lo_run = block_scan(lo_x, S.scratch, all);
    const bool exact = count || shift == 0;
    int last = -1;
    for (int q = 0; q < per; ++q) {
      hi_run += hw[q];
      lo_run += lw[q];
      if (hw[q] == 0) continue;
      last = b0 + q;
      if ((exact ? lo_run : hi_run + (hi_run >> 30)) >= goal) atomicMin(&S.lo, b0 + q);
      if ((exact ? lo_run : lo_run - (lo_run >> 30)) >= goal) atomicMin(&S.hi, b0 + q);
    }
    if (threadIdx.x == 0) S.above = -1;
    __syncthreads();
    if (last >= 0) atomicMax(&S.above, last);
    __syncthreads();
    const int end = S.above;
    const int hi = S.hi == INT_MAX ? end : S.hi;
    const int lo = S.lo == INT_MAX ? end : min(S.lo, hi);
    b.by_key = true;
    b.kmax = kmax - (static_cast<uint32_t>(lo) << shift);
    const uint32_t last_top = kmax - (static_cast<uint32_t>(hi) << shift);
    const uint32_t span = (1u << shift) - 1;
    b.kmin = last_top - kmin < span ? kmin : last_top - span;
    b.edge = key_value(b.kmin);
    __syncthreads();
  }

  // Cuts the set at the k-th token (count) or where the mass `target` is
  // reached, starting from a band of bins, and sets zc, ic.  `fin`: the last
  // cut, whose sums give the token as well (min-p's threshold zt is then
  // part of it).  False where min-p ends the kept tokens first: its cut is set,
  // its sums are not.
  __device__ bool cut(Band b, bool count, uint64_t goal, bool fin, float zt, const float* u) {
    for (int it = 0; it < 40; ++it) {  // (each turn shrinks the band; three are the usual most)
      if (fin && b.by_key && order_key(zt) > b.kmax) {
        zc = zt;
        ic = INT_MAX;
        return false;
      }
      gather(b, !count || (fin && u != nullptr));
      const int n = gathered();
      if (n <= kCap) {
        if (rank == 0) resolve(n, count, goal, fin, zt, u);
        publish();
        break;
      }
      if (rank == 0) {
        uint64_t w;
        int above, band;
        seg_totals(w, above, band);
        uint32_t lo = 0xffffffffu, hi = 0;
        for (int s = 0; s < C * kRowWarps; ++s) {
          lo = min(lo, S.segkmin[s]);
          hi = max(hi, S.segkmax[s]);
        }
        if (threadIdx.x == 0) {
          S.dec.kmin = lo;
          S.dec.kmax = hi;
          S.dec.kept = above;
          S.dec.W = w;
        }
        if (lo == hi) resolve_tie(band, above, w, key_value(lo), count, goal, fin, zt, u);
      }
      publish();
      b.kmin = S.dec.kmin;
      b.kmax = S.dec.kmax;
      if (b.kmin == b.kmax) {
        find_tie(key_value(b.kmin));
        break;
      }
      const uint64_t before = count ? static_cast<uint64_t>(S.dec.kept) : S.dec.W;
      __syncthreads();
      narrow(b, count, goal > before ? goal - before : 0);
    }
    zc = S.dec.zc;
    ic = S.dec.ic;
    return true;
  }

  __device__ __forceinline__ static float listed_logit(uint64_t k) { return key_value(~static_cast<uint32_t>(k >> 32)); }

  // Rank 0, the band collected: where the cut falls in it.  More keys than are
  // sorted quickly are first split into bins of their own.
  __device__ void resolve(int n, bool count, uint64_t goal, bool fin, float zt, const float* u) {
    uint64_t* list = reinterpret_cast<uint64_t*>(S.total);
    uint64_t w;
    int above, band;
    pull(n);
    seg_totals(w, above, band);
    if (count) w = above;
    uint64_t* sub = list;
    int m = n;
    if (n > kRowThreads / 2) {
      // bins of the keys' range, a thread's each: counts or masses
      uint64_t* bin = reinterpret_cast<uint64_t*>(S.hist);
      uint32_t lo = 0xffffffffu, hi = 0;
      for (int i = threadIdx.x; i < n; i += kRowThreads) {
        lo = min(lo, static_cast<uint32_t>(list[i] >> 32));
        hi = max(hi, static_cast<uint32_t>(list[i] >> 32));
      }
      lo = __reduce_min_sync(0xffffffffu, lo);
      hi = __reduce_max_sync(0xffffffffu, hi);
      bin[threadIdx.x] = 0;
      if (threadIdx.x == 0) {
        S.lo = INT_MAX;
        S.hi = 0;
      }
      if (lane == 0) S.scratch[warp] = (static_cast<uint64_t>(lo) << 32) | hi;
      __syncthreads();
      for (int x = 0; x < kRowWarps; ++x) {
        lo = min(lo, static_cast<uint32_t>(S.scratch[x] >> 32));
        hi = max(hi, static_cast<uint32_t>(S.scratch[x]));
      }
      int shift = 0;
      while (((hi - lo) >> shift) >= kRowThreads) ++shift;
      for (int i = threadIdx.x; i < n; i += kRowThreads)
        atomicAdd(reinterpret_cast<unsigned long long*>(&bin[(static_cast<uint32_t>(list[i] >> 32) - lo) >> shift]),
                  count ? 1ull : fixed_weight(listed_logit(list[i])));
      __syncthreads();
      const uint64_t mine = bin[threadIdx.x];
      uint64_t all;
      const uint64_t before = w + block_scan(mine, S.scratch, all);
      if (mine && before + mine >= goal) atomicMin(&S.lo, static_cast<int>(threadIdx.x));
      __syncthreads();
      const int at = S.lo == INT_MAX ? static_cast<int>((hi - lo) >> shift) : S.lo;
      if (static_cast<int>(threadIdx.x) == at) S.scratch[0] = before;
      __syncthreads();
      w = S.scratch[0];
      // the keys of that bin
      sub = reinterpret_cast<uint64_t*>(S.hist) + kRowThreads;
      for (int i = threadIdx.x; i < n; i += kRowThreads)
        if (static_cast<int>((static_cast<uint32_t>(list[i] >> 32) - lo) >> shift) == at) sub[atomicAdd(&S.hi, 1)] = list[i];
      __syncthreads();
      m = S.hi;
    }
    if (threadIdx.x == 0) {
      S.lo = m;
      S.above = 0;
    }
    sort(sub, m);
    constexpr int per = kCap / kRowThreads;
    const int i0 = threadIdx.x * per;
    uint64_t v[per], x = 0;
#pragma unroll
    for (int q = 0; q < per; ++q) {
      v[q] = i0 + q < m ? (count ? 1ull : fixed_weight(listed_logit(sub[i0 + q]))) : 0;
      x += v[q];
    }
    uint64_t all;
    uint64_t run = w + block_scan(x, S.scratch, all);
#pragma unroll
    for (int q = 0; q < per; ++q) {
      run += v[q];
      if (i0 + q < m && run >= goal) atomicMin(&S.lo, i0 + q);
    }
    __syncthreads();
    const uint64_t cutkey = sub[max(0, min(S.lo, m - 1))];
    float z = listed_logit(cutkey);
    int idx = static_cast<int>(cutkey & 0xffffffffu);
    if (fin && z < zt) {  // min-p ends the kept tokens earlier
      z = zt;
      idx = INT_MAX;
    }
    zc = z;
    ic = idx;
    // the band's tokens that the cut keeps
    int kept = 0;
    for (int i = threadIdx.x; i < n; i += kRowThreads)
      kept += in_set(listed_logit(list[i]), static_cast<int>(list[i] & 0xffffffffu));
    kept = __reduce_add_sync(0xffffffffu, kept);
    if (lane == 0 && kept) atomicAdd(&S.above, kept);
    __syncthreads();
    if (threadIdx.x == 0) {
      S.dec.tie_seg = -1;
      S.dec.zc = z;
      S.dec.ic = idx;
      S.dec.kept = above + S.above;
    }
    if (fin && u) finish(n, 0, 0.f, *u);
  }

  // Rank 0, every token down to the k-th's bin collected (n of them): top-k,
  // top-p and min-p on the sorted list.
  __device__ void resolve_top(int n, int k, float tp, float zt, const float* u) {
    uint64_t* list = reinterpret_cast<uint64_t*>(S.total);
    pull(n);
    sort(list, n);
    const int m = min(k, n);
    constexpr int per = kCap / kRowThreads;
    const int i0 = threadIdx.x * per;
    uint64_t v[per], x = 0;
#pragma unroll
    for (int q = 0; q < per; ++q) {
      v[q] = i0 + q < m ? fixed_weight(listed_logit(list[i0 + q])) : 0;
      x += v[q];
    }
    uint64_t all;
    uint64_t run = block_scan(x, S.scratch, all);
    uint64_t goal = tp < 1.f ? __umul64hi(all, __float2ull_rd(tp * 18446744073709551616.f)) + 1 : all;
    goal -= goal >> 36;  // kSlack
    if (threadIdx.x == 0) S.lo = m - 1;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < per; ++q) {
      run += v[q];
      if (i0 + q < m && (tp < 1.f && run >= goal)) atomicMin(&S.lo, i0 + q);
      if (i0 + q < m && i0 + q > 0 && listed_logit(list[i0 + q]) < zt) atomicMin(&S.lo, i0 + q - 1);
    }
    __syncthreads();
    const int last = S.lo;
    zc = listed_logit(list[last]);
    ic = static_cast<int>(list[last] & 0xffffffffu);
    if (threadIdx.x == 0) {
      S.dec.tie_seg = -1;
      S.dec.zc = zc;
      S.dec.ic = ic;
      S.dec.kept = last + 1;
    }
    if (u) finish(n, 0, 0.f, *u);
  }

  // Rank 0, a band of n > kCap equal logits: how many of them are kept, and
  // which segment holds the last one.
  __device__ void resolve_tie(int n, int above, uint64_t w, float z, bool count, uint64_t goal, bool fin, float zt,
                              const float* u) {
    const uint64_t before = count ? static_cast<uint64_t>(above) : w, one = count ? 1 : fixed_weight(z);
    const uint64_t left_over = goal > before ? goal - before : 0;
    int nb = static_cast<int>(min(max((left_over + one - 1) / one, uint64_t(1)), static_cast<uint64_t>(n)));
    if (fin && z < zt) nb = 0;
    if (threadIdx.x == 0) {
      S.dec.tie_seg = -1;
      S.dec.zc = nb > 0 ? z : zt;
      S.dec.ic = INT_MAX;
      S.dec.kept = above + nb;
      int left = nb;
      for (int s = 0; s < C * kRowWarps && left > 0; ++s) {
        if (S.segband[s] >= left) {
          S.dec.tie_seg = s;
          S.dec.tie_rank = left - 1;
          break;
        }
        left -= S.segband[s];
      }
    }
    __syncthreads();
    if (fin && u) finish(0, nb, z, *u);
  }

  // The index of the tie_rank-th logit equal to z in segment tie_seg, to
  // every CTA.
  __device__ void find_tie(float z) {
    const int ts = S.dec.tie_seg;
    __syncthreads();
    if (ts >= 0 && ts / kRowWarps == rank && ts % kRowWarps == warp) {
      int left = S.dec.tie_rank;
      bool found = false;
      for (int j0 = 0; j0 < sl.nv && !found; j0 += 32) {
        const int j = j0 + lane;
        float x[Elem<DT>::VW];
        int mine = 0;
        const int i0 = sl.base + (sl.v0 + j) * Elem<DT>::VW;
        if (j < sl.nv) {
          Elem<DT>::unpack(sl.data[sl.v0 + j], x);
#pragma unroll
          for (int q = 0; q < Elem<DT>::VW; ++q) mine += (x[q] == z && in_set(x[q], i0 + q));
        }
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        int at = left - (inc - mine);
        if (mine > 0 && at >= 0 && at < mine) {
#pragma unroll
          for (int q = 0; q < Elem<DT>::VW; ++q)
            if (x[q] == z && in_set(x[q], i0 + q) && at-- == 0)
              for (int r = 0; r < C; ++r) peer(&S.dec, r)->ic = i0 + q;
        }
        found = __any_sync(0xffffffffu, mine > 0 && left - (inc - mine) >= 0 && left - (inc - mine) < mine);
        left -= __shfl_sync(0xffffffffu, inc, 31);
      }
    }
    cluster_sync();
  }

  // Rank 0: total weight of the kept tokens, and the segment where the
  // running sum in index order passes u times it.  Kept: the segments' sums,
  // those of the n collected tokens that zc, ic keep, and the first nt logits
  // equal to z.
  __device__ void finish(int n_list, int nt, float z, float u) {
    const uint64_t* list = reinterpret_cast<const uint64_t*>(S.total);
    uint64_t* fix = reinterpret_cast<uint64_t*>(S.hist);  // free by now
    const int n = C * kRowWarps;
    __syncthreads();
    for (int s = threadIdx.x; s < n; s += kRowThreads) fix[s] = S.segsum[s];
    __syncthreads();
    for (int i = threadIdx.x; i < n_list; i += kRowThreads) {
      const float x = listed_logit(list[i]);
      const int idx = static_cast<int>(list[i] & 0xffffffffu);
      if (!in_set(x, idx)) continue;
      const int vec = idx / Elem<DT>::VW, cta = quotient(vec, split.svec);
      const int s = cta * kRowWarps + quotient(vec - cta * split.svec, split.gvec);
      atomicAdd(reinterpret_cast<unsigned long long*>(&fix[s]), draw_weight(x));
    }
    if (nt > 0 && threadIdx.x == 0) {
      const uint64_t one = draw_weight(z);
      for (int s = 0; s < n && nt > 0; ++s) {
        const int take = min(nt, S.segband[s]);
        fix[s] += one * static_cast<uint64_t>(take);
        nt -= take;
      }
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      const int per = (n + 31) / 32;
      uint64_t x = 0;
      for (int q = 0; q < per; ++q) x += lane * per + q < n ? fix[lane * per + q] : 0;
      uint64_t inc = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      const uint64_t all = __shfl_sync(0xffffffffu, inc, 31);
      // (whole numbers: run > u W exactly if run > its floor)
      uint64_t t = u > 0.f && u < 1.f ? __umul64hi(all, __float2ull_rd(u * 18446744073709551616.f)) : 0;
      t += t >> 36;  // kSlack
      const unsigned over = __ballot_sync(0xffffffffu, u < 1.f && inc > t);
      const unsigned some = __ballot_sync(0xffffffffu, x > 0);
      const bool fell = over == 0;
      const int who = fell ? 31 - __clz(some) : __ffs(over) - 1;
      if (lane == who) {
        uint64_t run = inc - x;
        int at = -1;
        uint64_t before = run;
        for (int q = 0; q < per; ++q) {
          const int s = lane * per + q;
          if (s >= n || fix[s] == 0) continue;
          at = s;
          before = run;
          run += fix[s];
          if (!fell && run > t) break;
        }
        S.dec.seg = at;
        S.dec.rem = fell ? ~0ull : t - before;
        S.dec.W = all;
        S.dec.fallback = fell;
      }
    }
    __syncthreads();
  }

  // a / b for 0 <= a < 2^24.
  __device__ __forceinline__ static int quotient(int a, int b) {
    int q = static_cast<int>(__fdividef(static_cast<float>(a), static_cast<float>(b)));
    q -= q * b > a;
    return q + ((q + 1) * b <= a);
  }
  RowSplit split;
};

// One row per cluster: the cut, the token, the filtered logits.
template <int DT>
__global__ void __launch_bounds__(kRowThreads, 2) sample_filter_kernel(const __grid_constant__ FilterParams P) {
  using E = Elem<DT>;
  extern __shared__ __align__(16) char smem[];
  __shared__ FilterShared S;
  const int C = P.sp.C, V = P.sp.V;
  const int rank = cluster_rank();
  const int64_t row = blockIdx.x / C;
  const int64_t b = row / P.R;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  cluster_arrive();  // waited for before the first remote write
  FilterRow<DT, false> F(S);
  F.rank = rank;
  F.C = C;
  F.V = V;
  F.lane = lane;
  F.warp = warp;
  F.split = P.sp;
  const char* zrow = reinterpret_cast<const char*>(P.z) + (b * P.bs + (row - b * P.R) * P.rs) * E::ES;
  F.sl.init(smem, P.sp, rank);
  F.sl.load(zrow, P.sp, &S.bars[warp]);
  for (int j = threadIdx.x; j < kGrid; j += kRowThreads) {
    S.tab.e[j] = P.tab.e[j];
    S.tab.p[j] = P.tab.p[j];
  }
  if (threadIdx.x == 0) S.above = 0;  // (this CTA's error bits, until the exchange)
  F.set_units();
  const float T = P.temp[b];
  const int k = P.top_k ? P.top_k[b] : 0;
  const float tp = P.top_p ? P.top_p[b] : 1.f;
  const float mp = P.min_p ? P.min_p[b] : 0.f;
  const float* u = P.u ? P.u + row : nullptr;
  int bad = 0;
  if (!(T >= 0.f) || T > 3.4e38f) bad |= kBadTemp;
  if (k < 0 || !(tp >= 0.f && tp <= 1.f) || !(mp >= 0.f && mp <= 1.f)) bad |= kBadFilter;
  // The row's scales in fp64, by one thread while the copies run.
  double tf = 0, tm = 0;
  if (threadIdx.x == 0) {
    const double Td = fmaxf(T, 1e-30f), lnf = -kWindow * 0.69314718055994530942;
    S.sc.set_factor<DT>(1.4426950408889634074 / Td);
    tf = Td * lnf;
    tm = mp > 0.f ? Td * fmax(log(static_cast<double>(mp)), lnf) : tf;
  }
  __syncthreads();
  if (!F.sl.load_wait(&S.bars[warp]) && lane == 0) atomicOr(&S.above, kTimeout);
  const float mc = block_max_nan(F.sl.warp_max(), S.fscratch);
  cluster_wait();
  push_all(S.xmax, rank, C, mc);
  push_all(S.xbad, rank, C, S.above);
  cluster_sync();
  float m = neg_inf();
  for (int r = 0; r < C; ++r) {
    m = max_nan(m, S.xmax[r]);
    bad |= S.xbad[r];
  }
  if (!(m > neg_inf() && m < pos_inf())) bad |= kNonFinite;

  F.zc = pos_inf();  // (nothing kept)
  F.ic = -1;
  bool pick = false;  // the token lies in S.dec's segment
  if (bad) {
    if (rank == 0 && threadIdx.x == 0) {
      if (P.tokens) P.tokens[row] = -1;
      if (P.prob) P.prob[row] = 0.f;
      if (P.kept) P.kept[row] = 0;
      if (P.status) P.status[row] = bad;
    }
  } else if (T == 0.f) {
    int first = INT_MAX;
    F.sl.each([&](float z, int i) {
      if (z == m) first = min(first, i);
    });
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) S.iscratch[warp] = first;
    __syncthreads();
    for (int w = 0; w < kRowWarps; ++w) first = min(first, S.iscratch[w]);
    push_all(S.xidx, rank, C, first);
    cluster_sync();
    for (int r = 0; r < C; ++r) first = min(first, S.xidx[r]);
    F.zc = m;
    F.ic = first;
    if (rank == 0 && threadIdx.x == 0) {
      if (P.tokens) P.tokens[row] = first;
      if (P.prob) P.prob[row] = 1.f;
      if (P.kept) P.kept[row] = 1;
      if (P.status) P.status[row] = 0;
    }
  } else {
    F.sc = S.sc;
    F.sc.set_max(m);
    if (threadIdx.x == 0) {
      S.zf = __double2float_ru(static_cast<double>(m) + tf);
      S.zt = fmaxf(S.zf, __double2float_ru(static_cast<double>(m) + tm));
    }
    F.clear_hist(kBins);  // (a barrier)
    const float zf = S.zf, zt = S.zt;
    F.zc = zf;
    F.ic = INT_MAX;
    const bool use_k = k > 0 && k < V, use_p = tp < 1.f;
    const int dt = zt > zf ? F.sc.template bin<false>(zt) : kBins;
    bool done = false;
    for (int stage = use_k ? 0 : 1; stage < (use_p ? 2 : 1); ++stage) {
      const bool count = stage == 0;
      if (!count && use_k) F.clear_hist(kBins);
      if (count) {
        F.sl.each([&](float z, int) {
          if (z >= zf) atomicAdd(&S.hist[F.sc.template bin<false>(z)], 1u);
        });
      } else {
        float low = 0.f;
        const float cut = F.zc;
        const int last = F.ic;
        auto add = [&](float z) {
          int d;
          uint32_t v;
          float e;
          F.sc.template weight<DT>(z, F.lin, F.inv, F.one, d, v, e);
          low += e;
          atomicAdd(&S.hist[d], v);
        };
        if (last == INT_MAX) {
          F.sl.each([&](float z, int) {
            if (z >= cut) add(z);
          });
        } else {
          F.sl.each([&](float z, int i) {
            if (z >= cut && F.in_set(z, i)) add(z);
          });
        }
        push_all(S.xsum, rank, C, F.block_sum_u(static_cast<uint64_t>(__float2ll_rn(low * F.unit))));
      }
      __syncthreads();
      F.merge(kBins);
      uint64_t goal = k;
      Band band;
      if (!(count ? F.template find_bins<true>(goal, 0.f, band) : F.template find_bins<false>(goal, tp, band)))
        continue;  // fewer than k
      if (count && S.before + static_cast<int>(S.total[band.hi]) <= kCap) {
        // few enough to collect: the rest is done on the list
        __syncthreads();
        band.lo = 0;
        F.gather(band, false);
        if (rank == 0) F.resolve_top(F.gathered(), k, tp, zt, u);
        F.publish();
        F.zc = S.dec.zc;
        F.ic = S.dec.ic;
        done = true;
        break;
      }
      const bool fin = !count || !use_p;
      if (fin && dt < band.lo) {  // min-p ends the kept tokens before the cut
        F.zc = zt;
        F.ic = INT_MAX;
        continue;
      }
      done = F.cut(band, count, goal, fin, zt, u) && fin;
    }
    if (!done) {  // no cut by bins: the tokens above min-p's threshold, if that is higher
      if (zt > F.zc) {
        F.zc = zt;
        F.ic = INT_MAX;
      }
      Band all;
      all.by_key = true;
      all.lo = all.hi = 0;
      all.kmin = all.kmax = 0;  // every token lies above
      all.edge = F.zc;
      F.gather(all, u != nullptr);
      if (rank == 0) {
        uint64_t w;
        int above, none;
        F.seg_totals(w, above, none);
        if (threadIdx.x == 0) S.dec.kept = above;
        if (u) F.finish(0, 0, 0.f, *u);
      }
      F.publish();
    }
    if (rank == 0 && threadIdx.x == 0) {
      if (P.kept) P.kept[row] = S.dec.kept;
      if (P.status) P.status[row] = (u && S.dec.fallback) ? kFallback : 0;
    }
    pick = u != nullptr && S.dec.seg / kRowWarps == rank && S.dec.seg % kRowWarps == warp;
  }

  if (pick) {  // one warp of the cluster
    const uint64_t rem = S.dec.rem;
    uint64_t run = 0;
    int last = -1, token = -1;
    float lastz = 0.f, tz = 0.f;
    for (int j0 = 0; j0 < F.sl.nv; j0 += 32) {
      const int j = j0 + lane;
      const int i0 = F.sl.base + (F.sl.v0 + j) * E::VW;
      float z[E::VW];
      uint64_t w[E::VW], x = 0;
      if (j < F.sl.nv) E::unpack(F.sl.data[F.sl.v0 + j], z);
#pragma unroll
      for (int q = 0; q < E::VW; ++q) {
        const bool in = j < F.sl.nv && F.in_set(z[q], i0 + q);
        w[q] = in ? F.draw_weight(z[q]) : 0;
        x += w[q];
        if (in) {
          last = i0 + q;
          lastz = z[q];
        }
      }
      uint64_t inc = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      const unsigned over = __ballot_sync(0xffffffffu, x > 0 && run + inc > rem);
      if (over) {
        const int who = __ffs(over) - 1;
        if (lane == who) {
          uint64_t y = run + inc;
#pragma unroll
          for (int q = E::VW - 1; q >= 0; --q) {  // the first whose sum passes: from the end
            if (w[q] > 0 && y > rem) {
              token = i0 + q;
              tz = z[q];
            }
            y -= w[q];
          }
        }
        token = __shfl_sync(0xffffffffu, token, who);
        tz = __shfl_sync(0xffffffffu, tz, who);
        break;
      }
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (token < 0) {  // the segment's last kept token
      const int most = __reduce_max_sync(0xffffffffu, last);
      const int who = __ffs(__ballot_sync(0xffffffffu, last == most)) - 1;
      token = most;
      tz = __shfl_sync(0xffffffffu, lastz, who);
    }
    if (lane == 0) {
      P.tokens[row] = token;
      if (P.prob) P.prob[row] = static_cast<float>(static_cast<double>(F.draw_weight(tz)) / static_cast<double>(S.dec.W));
    }
  }

  if (P.out) {
    char* orow = reinterpret_cast<char*>(P.out) + (b * P.obs + (row - b * P.R) * P.ors) * E::ES;
    for (int j0 = 0; j0 < F.sl.nv; j0 += 32) {
      const int j = j0 + lane, i0 = F.sl.base + (F.sl.v0 + j) * E::VW;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (j < F.sl.nv) {
        float z[E::VW];
        E::unpack(F.sl.data[F.sl.v0 + j], z);
#pragma unroll
        for (int q = 0; q < E::VW; ++q) z[q] = F.in_set(z[q], i0 + q) ? z[q] : neg_inf();
        w = pack_vec<DT>(z);
      }
      store_warp<DT>(orow, i0, V, j < F.sl.nv, w);
    }
  }
}

// One row per cluster: the k largest logits, in order, and the log-sum-exp.
template <int DT>
__global__ void __launch_bounds__(kRowThreads, 2) top_logits_kernel(const TopParams P) {
  using E = Elem<DT>;
  extern __shared__ __align__(16) char smem[];
  __shared__ FilterShared S;
  const int C = P.sp.C, V = P.sp.V, k = P.k;
  const int rank = cluster_rank();
  const int64_t row = blockIdx.x / C;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  cluster_arrive();
  FilterRow<DT, true> F(S);
  F.rank = rank;
  F.C = C;
  F.V = V;
  F.lane = lane;
  F.warp = warp;
  F.split = P.sp;
  const char* zrow = reinterpret_cast<const char*>(P.z) + row * P.rs * E::ES;
  F.sl.init(smem, P.sp, rank);
  F.sl.load(zrow, P.sp, &S.bars[warp]);
  if (threadIdx.x == 0) S.above = 0;
  __syncthreads();
  if (!F.sl.load_wait(&S.bars[warp]) && lane == 0) atomicOr(&S.above, kTimeout);
  const float mc = block_max_nan(F.sl.warp_max(), S.fscratch);
  cluster_wait();
  push_all(S.xmax, rank, C, mc);
  push_all(S.xbad, rank, C, S.above);
  cluster_sync();
  float m = neg_inf();
  int bad = 0;
  for (int r = 0; r < C; ++r) {
    m = max_nan(m, S.xmax[r]);
    bad |= S.xbad[r];
  }
  if (!(m > neg_inf() && m < pos_inf())) bad |= kNonFinite;
  if (bad) {
    if (rank == 0) {
      for (int j = threadIdx.x; j < k; j += kRowThreads) {
        P.ids[row * k + j] = -1;
        P.values[row * k + j] = neg_inf();
      }
      if (threadIdx.x == 0) {
        if (P.lse) P.lse[row] = __int_as_float(0x7fc00000);
        if (P.status) P.status[row] = bad;
      }
    }
    return;
  }
  F.sc.shift = m;  // (z - m keeps the order; exactness is of no matter here)
  F.sc.chi = 1.4426950f;
  F.sc.clo = 0.f;
  F.sc.gm = 0;
  F.zc = kNegMax;
  F.ic = INT_MAX;
  F.set_units();
  F.clear_hist(kBins);
  const float c = P.c;
  float s = 0.f;
  F.sl.each([&](float z, int) {
    s += ex2((z - m) * c);
    if (z >= kNegMax) atomicAdd(&S.hist[max(F.sc.template bin<true>(z), 0)], 1u);
  });
  s = warp_sum_f(s);
  if (lane == 0) S.fscratch[warp] = s;
  __syncthreads();
  s = 0.f;
  for (int w = 0; w < kRowWarps; ++w) s += S.fscratch[w];
  push_all(S.xexp, rank, C, s);
  __syncthreads();
  F.merge(kBins);
  Band band;
  uint64_t goal = k;
  const bool enough = F.template find_bins<true>(goal, 0.f, band);
  const int upto = enough ? S.before + static_cast<int>(S.total[band.hi]) : 0;
  __syncthreads();
  if (!enough) {
    band.by_key = false;
    band.hi = kBins - 1;
    band.edge = kNegMax;
  } else if (upto > kCap) {
    F.cut(band, true, k, false, kNegMax, nullptr);
    F.clear_hist(0);
    band.by_key = false;
    band.hi = kBins - 1;
    band.edge = F.zc;
  }
  band.lo = 0;
  F.gather(band, false);
  const int n = F.gathered();
  if (rank == 0) F.pull(n);
  cluster_sync();  // the other CTAs' lists have been read
  if (rank != 0) return;
  uint64_t* list = reinterpret_cast<uint64_t*>(S.total);
  F.sort(list, n);
  for (int j = threadIdx.x; j < k; j += kRowThreads) {
    P.ids[row * k + j] = j < n ? static_cast<int32_t>(list[j] & 0xffffffffu) : -1;
    P.values[row * k + j] = j < n ? key_value(~static_cast<uint32_t>(list[j] >> 32)) : neg_inf();
  }
  if (threadIdx.x == 0) {
    double t = 0;
    for (int r = 0; r < C; ++r) t += S.xexp[r];
    if (P.lse) P.lse[row] = static_cast<float>(static_cast<double>(m) * P.invT + log(t));
    if (P.status) P.status[row] = 0;
  }
}

}  // namespace specv
