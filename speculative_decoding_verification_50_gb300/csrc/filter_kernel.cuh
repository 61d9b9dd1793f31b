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
// Whole numbers come out of these sums (the cut, the token), so weights are
// pairs of fp32: 2^(E/64) from a table, exact to fp32, and the rest to first
// order apart, about 2^-30 relative together; totals are 64-bit integers in
// units of 2^-fbits of the largest weight (an SM does two fp64 operations a
// clock: a block's reductions in fp64 cost more than its passes over the row).  A
// sum in plain fp32 moves the cut of a flat distribution in one row of a
// hundred.
#pragma once

#include "distill_kernel.cuh"  // block_max_nan

namespace specv {

constexpr int kGrid = 64;                 // bins per unit of log2
constexpr int kWindow = 48;               // units below the maximum that carry weight
constexpr int kBins = kGrid * kWindow + 16;
constexpr int kCap = 2048;                // tokens sorted at once
constexpr int kBinsPerThread = (kBins + kRowThreads - 1) / kRowThreads;
constexpr int kBadFilter = 64;
constexpr float kMagic = 196608.f;        // 1.5 * 2^17: adding it rounds to 1/64
// Equal within 2^-36 counts as equal, so that sums of equal weights which meet
// a border exactly fall on its right side.
constexpr double kSlack = 1.4551915228366852e-11;

struct PairTable {
  float2 e[kGrid];  // 2^(j/64): (rounded to fp32, relative remainder)
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
  PairTable tab;
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

// The row's exponent scale: y = (z - shift) (chi + clo), Gm = the maximum's
// place on the grid of 1/64.
struct Scale {
  float shift, chi, clo;
  int gm;

  __device__ void set(float m, double c) {  // c = log2(e) / T
    chi = static_cast<float>(c);
    clo = static_cast<float>(c - static_cast<double>(chi));
    // |y| stays within the rounding trick's range; shifted logits are exact
    // where they carry weight (within 48 units of a maximum of 2^14 units).
    shift = fabsf(m) * chi > 16384.f ? m : 0.f;
    const float r = __fadd_rn(__fmul_rn(m - shift, chi), kMagic);
    gm = __float_as_int(r) - __float_as_int(kMagic);
  }
  // Distance from the maximum in bins (0 at the maximum).  CLAMP: for logits
  // that may lie anywhere below it (else: within the window).
  template <bool CLAMP>
  __device__ __forceinline__ int bin(float z) const {
    float p = __fmul_rn(z - shift, chi);
    if (CLAMP) p = fmaxf(p, -60000.f);
    const float r = __fadd_rn(p, kMagic);
    const int d = gm - (__float_as_int(r) - __float_as_int(kMagic));
    return CLAMP ? min(d, kBins - 1) : d;
  }
  // The weight 2^(y - gm/64) as h + l; d = its bin, g = what is left of y.
  __device__ __forceinline__ void weight(float z, const float2* tab, float& h, float& l, int& d, float& g) const {
    const float x = z - shift;
    const float p = __fmul_rn(x, chi);
    const float pe = fmaf(x, chi, -p);
    const float r = __fadd_rn(p, kMagic);
    g = __fadd_rn(p, -__fadd_rn(r, -kMagic)) + fmaf(x, clo, pe);
    const int e = __float_as_int(r) - __float_as_int(kMagic) - gm;
    d = -e;
    const float2 t = tab[e & (kGrid - 1)];
    h = __int_as_float(__float_as_int(t.x) + ((e >> 6) << 23));
    // 2^g - 1 for |g| <= 2^-7 (the next term is below 2^-34)
    l = h * fmaf(g, fmaf(g, fmaf(g, 0.05550411f, 0.24022651f), 0.69314718f), t.y);
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
  float2 tab[kGrid];
  uint32_t hist[kCap * 2];   // the CTA's histogram; in rank 0 the gathered keys (8 bytes each)
  uint32_t total[kBins];     // the row's histogram
  float xmax[kMaxCluster];
  uint64_t xsum[kMaxCluster];
  float xexp[kMaxCluster];
  int32_t xbad[kMaxCluster];
  int32_t xidx[kMaxCluster];
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
  uint64_t goal;
  Decision dec;
};
static_assert(kBins <= kCap * 2, "the histogram fits its array");

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
  float unit;   // 2^fbits

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
    const int per = (bins + C - 1) / C;
    const int b0 = rank * per, b1 = min(bins, b0 + per);
    for (int b = b0 + static_cast<int>(threadIdx.x); b < b1; b += kRowThreads) {
      uint32_t t = 0;
      for (int r = 0; r < C; ++r) t += peer(S.hist, r)[b];
      for (int r = 0; r < C; ++r) peer(S.total, r)[b] = t;
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
    for (int b = threadIdx.x; b < bins; b += kRowThreads) S.hist[b] = 0;
    if (threadIdx.x == 0) {
      S.ngather = 0;
      S.lo = S.hi = INT_MAX;
    }
    __syncthreads();
  }

  // Gathers the band's tokens at rank 0 and leaves, per segment, the number
  // and (sums) the weight of the tokens above the band, and the band's count
  // and range of keys.  Ends with a cluster barrier.
  __device__ void gather(const Band& b, bool sums) {
    PairSum acc;
    int above = 0, band = 0;
    uint32_t kmin = 0xffffffffu, kmax = 0;
    uint64_t* list = reinterpret_cast<uint64_t*>(peer(S.hist, 0));
    int* counter = peer(&S.ngather, 0);
    const float edge = b.edge;
    for (int j0 = 0; j0 < sl.nv; j0 += 32) {
      const int j = j0 + lane;
      float z[Elem<DT>::VW];
      if (j < sl.nv) {
        Elem<DT>::unpack(sl.data[sl.v0 + j], z);
      } else {
#pragma unroll
        for (int k = 0; k < Elem<DT>::VW; ++k) z[k] = neg_inf();
      }
      const int i0 = sl.base + (sl.v0 + j) * Elem<DT>::VW;
#pragma unroll
      for (int k = 0; k < Elem<DT>::VW; ++k) {
        const bool cand = z[k] >= edge && in_set(z[k], i0 + k);
        if (!__any_sync(0xffffffffu, cand)) continue;
        const int pl = cand ? place(z[k], b) : 2;
        if (pl == 0) {
          ++above;
          if (sums) {
            float h, l, g;
            int d;
            sc.weight(z[k], S.tab, h, l, d, g);
            acc.add(h, l);
          }
        }
        const unsigned in = __ballot_sync(0xffffffffu, pl == 1);
        if (in) {
          int pos = 0;
          if (lane == __ffs(in) - 1) pos = atomicAdd(counter, __popc(in));
          pos = __shfl_sync(0xffffffffu, pos, __ffs(in) - 1) + __popc(in & ((1u << lane) - 1));
          if (pl == 1) {
            ++band;
            const uint32_t key = order_key(z[k]);
            kmin = min(kmin, key);
            kmax = max(kmax, key);
            if (pos < kCap) list[pos] = (static_cast<uint64_t>(~key) << 32) | static_cast<uint32_t>(i0 + k);
          }
        }
      }
    }
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
    cluster_sync();
  }

  // Sorts rank 0's gathered keys ascending: logit descending, index ascending.
  __device__ void sort(int n) {
    uint64_t* list = reinterpret_cast<uint64_t*>(S.hist);
    int P = 2;
    while (P < n) P <<= 1;
    for (int i = n + static_cast<int>(threadIdx.x); i < P; i += kRowThreads) list[i] = ~0ull;
    __syncthreads();
    for (int size = 2; size <= P; size <<= 1)
      for (int step = size >> 1; step > 0; step >>= 1) {
        for (int t = threadIdx.x; t < P / 2; t += kRowThreads) {
          const int i = 2 * t - (t & (step - 1)), j = i + step;
          const uint64_t x = list[i], y = list[j];
          if ((x > y) == ((i & size) == 0)) {
            list[i] = y;
            list[j] = x;
          }
        }
        __syncthreads();
      }
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

  // A bin's mass, v counted in 2^-bits of its scale 2^(-d/64).
  __device__ __forceinline__ uint64_t mass(uint32_t v, int d, int bits) const {
    const uint32_t t = (__float_as_uint(S.tab[(-d) & (kGrid - 1)].x) << 8) | 0x80000000u;  // 2^31 2^(j/64)
    const int s = bits + 31 - fbits - ((-d) >> 6);
    const uint64_t x = static_cast<uint64_t>(v) * t;
    return s >= 64 ? 0 : s >= 0 ? x >> s : x << -s;
  }

  // Bins -> the band between the first bin where the cut may lie and the
  // first where it must.  COUNT: the goal-th token; else the mass `goal`, the
  // bins' masses being good to 2^-bits.  S.before: the count before the band.
  // False if the set ends before the goal-th token.
  template <bool COUNT>
  __device__ bool find_bins(uint64_t goal, int bits, Band& b) {
    const int b0 = threadIdx.x * kBinsPerThread;
    uint64_t v[kBinsPerThread], x = 0;
#pragma unroll
    for (int q = 0; q < kBinsPerThread; ++q) {
      const uint32_t n = b0 + q < kBins ? S.total[b0 + q] : 0u;
      v[q] = COUNT ? n : mass(n, b0 + q, bits);
      x += v[q];
    }
    uint64_t all;
    uint64_t run = block_scan(x, S.scratch, all);
    if (COUNT && all < goal) return false;
#pragma unroll
    for (int q = 0; q < kBinsPerThread; ++q) {
      const uint64_t before = run;
      run += v[q];
      const uint64_t slack = COUNT ? 0 : (run >> bits) + 1;
      if (v[q] && run + slack >= goal) {
        if (COUNT && before < goal) S.before = static_cast<int32_t>(before);
        atomicMin(&S.lo, b0 + q);
      }
      if (v[q] && run - slack >= goal) {
        atomicMin(&S.hi, b0 + q);
        break;
      }
    }
    __syncthreads();
    b.by_key = false;
    b.lo = S.lo == INT_MAX ? kBins - 1 : S.lo;
    b.hi = S.hi == INT_MAX ? kBins - 1 : S.hi;
    // 64 y >= gm - hi - 1/2 for every token of the band, with room for rounding
    const float e = sc.shift + (static_cast<float>(sc.gm - b.hi) - 0.5f) / (static_cast<float>(kGrid) * sc.chi);
    b.edge = b.hi >= kBins - 1 ? kNegMax : fmaxf(e - 1e-6f * (fabsf(e) + fabsf(sc.shift)) - 1e-30f, kNegMax);
    __syncthreads();
    return true;
  }

  __device__ uint64_t fixed_weight(float z) const {
    float h, l, g;
    int d;
    sc.weight(z, S.tab, h, l, d, g);
    return static_cast<uint64_t>(__float2ll_rn(h * unit) + __float2ll_rn(l * unit));
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
      const int n = *peer(&S.ngather, 0);
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

  // Rank 0, the band gathered: where the cut falls in it.
  __device__ void resolve(int n, bool count, uint64_t goal, bool fin, float zt, const float* u) {
    uint64_t* list = reinterpret_cast<uint64_t*>(S.hist);
    uint64_t w;
    int above, band;
    seg_totals(w, above, band);
    sort(n);
    if (threadIdx.x == 0) S.lo = S.hi = n;
    __syncthreads();
    int nb;
    if (count) {
      nb = min(static_cast<int>(goal) - above, n);
    } else {
      constexpr int per = kCap / kRowThreads;
      const int i0 = threadIdx.x * per;
      uint64_t v[per], x = 0;
#pragma unroll
      for (int q = 0; q < per; ++q) {
        v[q] = i0 + q < n ? fixed_weight(key_value(~static_cast<uint32_t>(list[i0 + q] >> 32))) : 0;
        x += v[q];
      }
      uint64_t all;
      uint64_t run = w + block_scan(x, S.scratch, all);
#pragma unroll
      for (int q = 0; q < per; ++q) {
        run += v[q];
        if (i0 + q < n && run >= goal) atomicMin(&S.lo, i0 + q);
      }
      __syncthreads();
      nb = min(S.lo + 1, n);
    }
    if (fin) {  // min-p may end the kept tokens earlier
      for (int i = threadIdx.x; i < n; i += kRowThreads)
        if (key_value(~static_cast<uint32_t>(list[i] >> 32)) < zt) atomicMin(&S.hi, i);
      __syncthreads();
      nb = min(nb, S.hi);
    }
    if (threadIdx.x == 0) {
      S.dec.tie_seg = -1;
      if (nb > 0) {
        S.dec.zc = key_value(~static_cast<uint32_t>(list[nb - 1] >> 32));
        S.dec.ic = static_cast<int32_t>(list[nb - 1] & 0xffffffffu);
      } else {
        S.dec.zc = zt;
        S.dec.ic = INT_MAX;
      }
      S.dec.kept = above + nb;
    }
    if (fin && u) finish(nb, 0, 0.f, *u);
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
  // the first nb gathered tokens, and the first nt logits equal to z.
  __device__ void finish(int nb, int nt, float z, float u) {
    const uint64_t* list = reinterpret_cast<const uint64_t*>(S.hist);
    uint64_t* fix = reinterpret_cast<uint64_t*>(S.total);  // free by now
    const int n = C * kRowWarps;
    __syncthreads();
    for (int s = threadIdx.x; s < n; s += kRowThreads) fix[s] = S.segsum[s];
    __syncthreads();
    const int seg = sl_segment_size();
    for (int i = threadIdx.x; i < nb; i += kRowThreads) {
      const float x = key_value(~static_cast<uint32_t>(list[i] >> 32));
      const int idx = static_cast<int>(list[i] & 0xffffffffu);
      const int cta = idx / cta_size();
      const int s = cta * kRowWarps + (idx - cta * cta_size()) / seg;
      atomicAdd(reinterpret_cast<unsigned long long*>(&fix[s]), fixed_weight(x));
    }
    if (nt > 0 && threadIdx.x == 0) {
      const uint64_t one = fixed_weight(z);
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
      const uint64_t t =
          __double2ull_rd(fmax(static_cast<double>(u), 0.0) * static_cast<double>(all) * (1.0 + kSlack));
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

  __device__ int cta_size() const { return split.svec * Elem<DT>::VW; }
  __device__ int sl_segment_size() const { return split.gvec * Elem<DT>::VW; }
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
  for (int j = threadIdx.x; j < kGrid; j += kRowThreads) S.tab[j] = P.tab.e[j];
  if (threadIdx.x == 0) S.above = 0;  // (this CTA's error bits, until the exchange)
  F.fbits = min(44, 62 - (32 - __clz(V)));
  F.unit = __int_as_float((127 + F.fbits) << 23);
  const float T = P.temp[b];
  const int k = P.top_k ? P.top_k[b] : 0;
  const float tp = P.top_p ? P.top_p[b] : 1.f;
  const float mp = P.min_p ? P.min_p[b] : 0.f;
  const float* u = P.u ? P.u + row : nullptr;
  int bad = 0;
  if (!(T >= 0.f) || T > 3.4e38f) bad |= kBadTemp;
  if (k < 0 || !(tp >= 0.f && tp <= 1.f) || !(mp >= 0.f && mp <= 1.f)) bad |= kBadFilter;
  // The row's scales in fp64, by one thread while the copies run.
  double c = 0, tf = 0, tm = 0;
  if (threadIdx.x == 0) {
    const double Td = fmaxf(T, 1e-30f), lnf = -kWindow * 0.69314718055994530942;
    c = 1.4426950408889634074 / Td;
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
    if (threadIdx.x == 0) {
      S.sc.set(m, c);
      S.zf = __double2float_ru(static_cast<double>(m) + tf);
      S.zt = fmaxf(S.zf, __double2float_ru(static_cast<double>(m) + tm));
    }
    __syncthreads();
    F.sc = S.sc;
    const float zf = S.zf, zt = S.zt;
    F.zc = zf;
    F.ic = INT_MAX;
    const bool use_k = k > 0 && k < V, use_p = tp < 1.f;
    const int dt = zt > zf ? F.sc.template bin<false>(zt) : kBins;
    bool done = false;
    // the shift that lets a bin hold every token's mass in 32 bits
    const int bits = min(14, 31 - (32 - __clz(V)));
    for (int stage = use_k ? 0 : 1; stage < (use_p ? 2 : 1); ++stage) {
      const bool count = stage == 0;
      F.clear_hist(kBins);
      PairSum acc;
      const float one = ldexpf(1.f, bits), lin = one * 0.69314718f;
      F.sl.each([&](float z, int i) {
        if (F.in_set(z, i)) {
          if (count) {
            atomicAdd(&S.hist[min(static_cast<unsigned>(F.sc.template bin<false>(z)), kBins - 1u)], 1u);
          } else {
            float h, l, g;
            int d;
            F.sc.weight(z, S.tab, h, l, d, g);
            acc.add(h, l);
            atomicAdd(&S.hist[min(static_cast<unsigned>(d), kBins - 1u)], static_cast<uint32_t>(__float2int_rn(fmaf(g, lin, one))));
          }
        }
      });
      if (!count) push_all(S.xsum, rank, C, F.block_sum_u(acc.fixed(F.unit)));
      __syncthreads();
      F.merge(kBins);
      uint64_t goal = k;
      if (!count) {
        if (threadIdx.x == 0) {
          uint64_t Z = 0;
          for (int r = 0; r < C; ++r) Z += S.xsum[r];
          S.goal = __double2ull_ru(static_cast<double>(tp) * static_cast<double>(Z) * (1.0 - kSlack));
        }
        __syncthreads();
        goal = S.goal;
      }
      Band band;
      if (!(count ? F.template find_bins<true>(goal, bits, band) : F.template find_bins<false>(goal, bits, band)))
        continue;  // fewer than k
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
        w[q] = in ? F.fixed_weight(z[q]) : 0;
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
      if (P.prob) P.prob[row] = static_cast<float>(static_cast<double>(F.fixed_weight(tz)) / static_cast<double>(S.dec.W));
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
  F.fbits = 0;
  F.unit = 1.f;
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
  if (!F.template find_bins<true>(k, 0, band)) {
    band.by_key = false;
    band.hi = kBins - 1;
    band.edge = kNegMax;
  } else if (S.before + S.total[band.hi] > kCap) {
    F.cut(band, true, k, false, kNegMax, nullptr);
    F.clear_hist(0);
    cluster_sync();
    band.by_key = false;
    band.hi = kBins - 1;
    band.edge = F.zc;
  }
  band.lo = 0;
  F.gather(band, false);
  if (rank != 0) return;  // (nothing of the other CTAs is read from here on)
  const int n = S.ngather;
  F.sort(n);
  const uint64_t* list = reinterpret_cast<const uint64_t*>(S.hist);
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
