// Sampling with temperature, top-k, top-p and min-p, and the k largest logits.
//
// A row's kept set is a prefix of its tokens in the order (logit descending,
// index ascending), so it is named by one logit and one index: kept iff
// z > zc, or z == zc and index <= ic.  The cut is found by a histogram of
// y = z log2(e) / T in bins of 1/32 below the maximum (counts for top-k, masses
// for top-p), which names the bin that the cut lies in; that band's tokens are
// collected, split or sorted, and summed exactly.  A band too full to collect
// is narrowed by the bits of the logits, then (all equal) by index.
//
// Whole numbers come out of the sums of weights 2^(y - max) (the cut, the
// token), and a sum in plain fp32 moves the cut of a flat distribution in one
// row of a hundred.  So a weight is 2^(-d/32) v 2^-28, d its bin and v a whole
// number (good to 2^-29, random): the bins sum v exactly, in two halves of 14
// bits (of up to 250,000 logits per part), and totals are 64-bit integers in
// units of 2^-fbits of the largest weight.  (An SM does two fp64 operations a
// clock: a block's reductions in fp64 cost more than its passes over the row.
// One 64-bit shared atomic a logit takes 56 clocks a warp where the two of 32
// bits take 6.6.)
#pragma once

#include "distill_kernel.cuh"  // block_max_nan

namespace specv {

constexpr int kGrid = 32;                 // bins per unit of log2
constexpr int kWindow = 48;               // units below the maximum that carry weight
constexpr int kBins = kGrid * kWindow + 16;
constexpr int kHead = 8 * kGrid;          // bins above a guessed maximum
constexpr int kHist = kBins + kHead;      // of a CTA's histogram
constexpr int kCap = 1536;                // tokens of a band that are worked on as a list
constexpr int kMaxBinned = 250000;        // logits of a CTA, so that a bin's halves fit 32 bits
constexpr int kMaxParts = 16;             // parts of a row that are summed apart: C * H
constexpr int kMaxH = 4;
constexpr int kBadFilter = 64;
constexpr float kMagic = 393216.f;        // 1.5 * 2^18: adding it rounds to 1/32
// Sums equal within 2^-36 (x >> 36) count as equal, so that equal weights which
// meet a border exactly fall on its right side.
constexpr int kSlack = 36;
// The threads' maxima bound the k-th largest logit where there are at least
// this many of them per token wanted (their k-th is then exceeded by about
// 1.15 k logits).  Against a histogram of every logit (us): the 256 largest of
// 2048 x 152064 bf16 236, 366; of 64 rows 21, 27; 100 of 333 x 50257 fp32 47, 61.
constexpr int kFewTop = 4;

struct BinTable {
  uint64_t e[kGrid];  // 2^(63 + j/32)
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
// A collected token: ascending is logit descending, index ascending.
__device__ __forceinline__ uint64_t token_key(float z, int i) {
  return (static_cast<uint64_t>(~order_key(z)) << 32) | static_cast<uint32_t>(i);
}
__device__ __forceinline__ float token_logit(uint64_t k) { return key_value(~static_cast<uint32_t>(k >> 32)); }
__device__ __forceinline__ int token_index(uint64_t k) { return static_cast<int>(k & 0xffffffffu); }

__device__ __forceinline__ uint64_t warp_sum_u(uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// a x for 0 <= a < 1, rounded down.
__device__ __forceinline__ uint64_t fraction(float a, uint64_t x) {
  return __umul64hi(x, __float2ull_rd(a * 18446744073709551616.f));
}

// The row's exponent scale: y = (z - shift) (chi + clo), gm = the maximum's
// place on the grid of 1/32.  Weights are relative to 2^(gm / 32).
struct Scale {
  float shift, chi, clo;
  int gm;

  // chi + clo = log2(e) / T, to about 2^-47.
  __device__ void set_factor(float T) {
    chi = __fdiv_rn(1.44269502f, T);  // log2(e) = 1.44269502 + 1.925963e-8
    clo = __fdiv_rn(fmaf(-chi, T, 1.44269502f) + 1.925963e-8f, T);
  }
  __device__ void set_max(float m) {
    // |y| stays within the rounding trick's range; shifted logits are exact
    // where they carry weight (within 48 units of a maximum of 2^14 units).
    shift = fabsf(m) * chi > 16384.f ? m : 0.f;
    gm = place(m - shift);
  }
  // x chi on the grid, as bits above those of 0 (rounding is monotone).
  __device__ __forceinline__ int place(float x) const { return __float_as_int(fmaf(x, chi, kMagic)) - __float_as_int(kMagic); }
  // Distance from the maximum in bins: 0 <= bin <= 48 * 32 + 3 for a logit of
  // the window.  CLAMP: for any logit below the maximum.
  template <bool CLAMP>
  __device__ __forceinline__ int bin(float z) const {
    if (!CLAMP) return gm - place(z - shift);
    const float r = fmaxf(fmaf(z - shift, chi, kMagic), kMagic - 60000.f);
    return min(gm + __float_as_int(kMagic) - __float_as_int(r), kBins - 1);
  }
  // v of a logit of the window, and its place on the grid with the bits of 0's.
  // SHIFT false: shift is 0.
  template <bool SHIFT>
  __device__ __forceinline__ uint32_t weight_at(float z, int& at) const {
    const float x = SHIFT ? z - shift : z;
    const float r = fmaf(x, chi, kMagic);
    at = __float_as_int(r);
    const float g = fmaf(x, clo, fmaf(x, chi, kMagic - r));  // to 2^-30
    // 2^28 (2^g - 1) for |g| <= 2^-6 (the next term is below 2^-39), rounded to a
    // whole number by adding 1.5 * 2^23
    const float t = fmaf(g * 268435456.f, fmaf(g, fmaf(g, fmaf(g, 0.009618129f, 0.05550411f), 0.24022651f), 0.69314718f),
                         12582912.f);
    return __float_as_uint(t) - (0x4b400000u - 0x10000000u);
  }
  // v and d of a logit of the window.
  __device__ __forceinline__ uint32_t weight(float z, int& d) const {
    int at;
    const uint32_t v = weight_at<true>(z, at);
    d = gm + __float_as_int(kMagic) - at;
    return v;
  }
  // A logit that every logit of bins <= d is at or above, with room for
  // rounding (side -1); that every logit at or above it has a bin < d (+1).
  __device__ __forceinline__ float edge(int d, int side) const {
    const float e = shift + (static_cast<float>(gm - d) + 0.5f * static_cast<float>(side)) / (static_cast<float>(kGrid) * chi);
    const float room = 1e-6f * (fabsf(e) + fabsf(shift)) + 1e-30f;
    return side < 0 ? fmaxf(e - room, kNegMax) : e + room;
  }
};

// What rank 0 decides and every CTA reads.
struct Decision {
  float zc;
  int32_t ic;
  int32_t kept;
  int32_t fallback;
  int32_t tie_part, tie_rank; // -1, or where the last kept of many equal logits lies
  int32_t part;               // -1, or the part that the token is to be drawn from
  int32_t token;              // the token, if rank 0 has it (part = -1)
  uint64_t rem;               // u W less what lies before that part
  uint64_t W;
  float z;                    // the token's logit
};

struct FilterShared {
  uint64_t bars[kRowWarps * kMaxRing];
  uint64_t tab[kGrid];
  uint32_t tab32[kGrid];     // its upper halves, rounded
  float total[kBins];        // the row's histogram; then, in rank 0, bins of the list
  uint64_t Z;                // the row's weight
  // one value per CTA, pushed to every CTA (xmass, xband: per part)
  uint64_t xmass[kMaxParts];
  int32_t xband[kMaxParts];
  float xmax[kMaxCluster], xexp[kMaxCluster];
  int32_t xbad[kMaxCluster], xidx[kMaxCluster], xabove[kMaxCluster], xcount[kMaxCluster];
  uint32_t xkmin[kMaxCluster], xkmax[kMaxCluster];
  // within a CTA
  uint64_t scratch[kRowWarps];
  float fscratch[kRowWarps];
  int32_t iscratch[kRowWarps];
  uint64_t mine[kMaxH];      // per part: the weight in the bins before the band
  uint64_t mass[kMaxH];      // per part: of tokens above the band that share its bins
  int32_t band[kMaxH];       // per part: the band's tokens
  int32_t above, ncollect, kept, bad;
  uint32_t fix32[3][kMaxParts];  // per part, in pieces of 15 bits
  uint32_t kmin, kmax;
  uint32_t upper;            // a band that is a lower half: the upper one's largest key
  int32_t lo, hi;
  int32_t before;
  float zf, zt;
  Decision dec;
};
static_assert(2 * kBins <= 4 * kCap && 2 * kRowThreads <= kBins, "arrays that share memory fit");

// Bytes of a CTA's work space, behind the held vectors: its parts' histograms
// (two halves each); then the band's tokens that it collects, and in rank 0,
// behind them, those of all CTAs.
__host__ __device__ constexpr int work_bytes(int H) {
  return H * 2 * kHist * 4 > 2 * kCap * 8 ? H * 2 * kHist * 4 : 2 * kCap * 8;
}

// The part of the set that the cut lies in: bins [lo, hi], by keys [kmin, kmax]
// of them once it has been narrowed.  Tokens above it are certainly kept by the
// cut, those below certainly not.
struct Band {
  bool by_key;
  int lo, hi;
  float elo, ehi;        // the bins' logits lie in [elo, ehi) (the keys' from elo on)
  uint32_t kmin, kmax;
};

// kGiven: at min-p's threshold.
enum CutKind { kByCount, kByMass, kGiven };

template <int DT, bool CLAMP>
struct FilterRow {
  FilterShared& S;
  using Slice = RowSlice<DT, false, CLAMP>;
  Slice sl;
  const RowSplit& split;  // (of the launch's arguments: no registers)
  const int &C, &V, &H;
  Scale sc;
  char* smem;        // the held vectors
  uint64_t* work;
  int rank, lane, warp;
  int sub;           // the part of the CTA's slice that this warp's segment belongs to
  float zc;
  int ic;
  int off;    // the histograms' bin of the maximum
  int fbits;  // sums are in units of 2^-fbits, so that V weights stay below 2^62

  __device__ FilterRow(FilterShared& s, const RowSplit& sp, char* shared, const void* z)
      : S(s), split(sp), C(sp.C), V(sp.V), H(sp.H), smem(shared), rank(cluster_rank()), lane(threadIdx.x & 31), warp(threadIdx.x >> 5) {
    work = reinterpret_cast<uint64_t*>(smem + row_bytes(sp.rvec, 0));
    sub = warp * sp.H / kRowWarps;
    sl.init(smem, S.bars, sp, z, rank, warp);
    off = 0;
    fbits = min(44, 62 - (32 - __clz(V)));
  }

  __device__ __forceinline__ int shift_H() const { return H >> 1; }  // log2 of 1, 2, 4
  __device__ uint32_t* hist(int part) const { return reinterpret_cast<uint32_t*>(work) + part * (2 * kHist) + off; }
  __device__ uint64_t* own_list() const { return work; }
  __device__ uint64_t* list() const { return work + kCap; }

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

  // v 2^-28 2^(-d/32) in units of 2^-fbits; v < 2^28 V.
  __device__ __forceinline__ uint64_t mass(uint64_t v, int d) const {
    const uint64_t x = __umul64hi(v << (fbits - 27), S.tab[(-d) & (kGrid - 1)]);
    const int s = (d + kGrid - 1) / kGrid;
    return s > 0 ? (x + (1ull << (s - 1))) >> s : x;
  }
  // A token's weight in whole units, at least one, so that every kept token can
  // be drawn: what light tokens lose or gain by that, a unit each, is the draw's
  // resolution.  (A list's and a part's tokens; the histograms' masses take the
  // exact product.)
  __device__ __forceinline__ uint64_t weight(float z) const {
    int d;
    const uint32_t v = sc.weight(z, d);
    const uint64_t x = static_cast<uint64_t>(v) * S.tab32[(-d) & (kGrid - 1)];
    const int s = min(58 - fbits + ((d + kGrid - 1) >> 5), 62);
    return max(((x >> s) + 1) >> 1, uint64_t(1));
  }

  // A token's share of W, from its logit: 2^-29 of itself whatever its weight.
  __device__ float share(float z, uint64_t W) const {
    int d;
    const uint32_t v = sc.weight(z, d);
    const double w = static_cast<double>(v) * static_cast<double>(S.tab[(-d) & (kGrid - 1)]);
    const double unit = __hiloint2double((1023 + fbits - 91 - ((d + kGrid - 1) >> 5)) << 20, 0);  // a power of two
    return static_cast<float>(w * unit / static_cast<double>(W));
  }

  // The cluster's barrier.
  __device__ __forceinline__ void sync_all() const {
    if (C == 1) __syncthreads();
    else cluster_sync();
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
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) {
      const T y = scratch[w];
      if (w < warp) base += y;
      all += y;
    }
    return base + inc - x;
  }

  // Block-wide sum (every thread gets it).
  __device__ uint64_t block_sum_u(uint64_t x) {
    x = warp_sum_u(x);
    __syncthreads();
    if (lane == 0) S.scratch[warp] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) x += S.scratch[w];
    return x;
  }

  // A logit's weight into this warp's histogram, if z >= cut and `also`: `base`,
  // the shared address of the bin whose place has bits 0; places above `most`
  // count as that one.  (Computed for every logit, only the additions under a
  // predicate: as a branch the compiler guarded each logit's arithmetic.)
  template <bool SHIFT>
  __device__ __forceinline__ void add_mass(uint32_t base, int most, float z, float cut, bool also) const {
    int at;
    const uint32_t v = sc.template weight_at<SHIFT>(z, at);
    const uint32_t bin = base - 4u * static_cast<uint32_t>(min(at, most));
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %6, 0;\n\tsetp.ge.and.f32 p, %1, %2, q;\n\t"
        "@p red.shared.add.u32 [%0], %3;\n\t@p red.shared.add.u32 [%0 + %5], %4;\n\t}"
        :: "r"(bin), "f"(z), "f"(cut), "r"(v >> 14), "r"(v & 0x3fffu), "n"(4 * kHist), "r"(static_cast<uint32_t>(also))
        : "memory");
  }
  __device__ __forceinline__ int most() const { return sc.gm + __float_as_int(kMagic) + off; }
  __device__ __forceinline__ uint32_t base() const {
    return static_cast<uint32_t>(__cvta_generic_to_shared(hist(sub))) +
           4u * static_cast<uint32_t>(sc.gm + __float_as_int(kMagic));
  }

  // A guess at the row's maximum, the same in every CTA: over the first vectors
  // of every warp's segment.  (cluster_wait has been called.)
  __device__ float guess_max() {
    float m = neg_inf();
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (lane + 32 * u < sl.nv) m = vec_max<DT>(sl.fetch(lane + 32 * u), m);
    m = block_max_nan(m, S.fscratch);
    push_all(S.xexp, rank, C, m);
    sync_all();
    m = neg_inf();
    for (int r = 0; r < C; ++r) m = max_nan(m, S.xexp[r]);
    return m;
  }

  // The first pass over a row, from memory (with a pass for the maximum before that for
  // the masses 2304 x 152064 fp32 take 7 % longer): the maximum, and on the way the
  // masses by bins below a guessed one (`sc`, without a shift; the first kHead bins are for
  // logits above it).  The guess holds if the maximum turns out to lie there, on the same
  // scale.
  __device__ float max_and_masses(float cut) {
    constexpr int VW = Elem<DT>::VW;
    using Vec = typename Elem<DT>::Vec;
    const uint32_t to = base();
    const int top = most();
    float m = neg_inf();
    sl.groups([&](const Vec(&x)[2], int) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        m = vec_max<DT>(x[u], m);
        float z[VW];
        Elem<DT>::unpack(x[u], z);
#pragma unroll
        for (int k = 0; k < VW; ++k)
          add_mass<false>(to, top, z[k], cut, true);
      }
    }, true);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
  }

  // Empty histograms and no tokens collected.  Ends with a barrier.
  __device__ void clear() {
    for (int b = threadIdx.x; b < H * (kHist / 2); b += kRowThreads)
      reinterpret_cast<uint4*>(work)[b] = make_uint4(0u, 0u, 0u, 0u);
    if (threadIdx.x < kMaxH) {
      S.mass[threadIdx.x] = 0;
      S.band[threadIdx.x] = 0;
    }
    if (threadIdx.x == 0) {
      S.Z = 0;
      S.above = S.ncollect = 0;
      S.kmin = 0xffffffffu;
      S.kmax = 0;
      S.upper = 0;
      S.lo = S.hi = INT_MAX;
    }
    __syncthreads();
  }

  // The row's histogram into S.total on every CTA, as counts or (MASS) masses,
  // whose exact sum goes to S.Z.  Each CTA adds up a share of the bins over the
  // cluster's parts.  Barriers: the cluster's, twice.
  // `last`: the last bin that counts.
  template <bool MASS>
  __device__ void merge(int bins, int last = kBins) {
    sync_all();
    const int per = (bins + C - 1) / C, parts = C * H;
    const int b0 = rank * per, b1 = min(bins, b0 + per);
    for (int b = b0 + warp * 32; b < b1; b += kRowThreads) {
      const int d = b + lane;
      const bool on = d < b1;
      uint64_t v = 0;
      for (int p0 = 0; p0 < parts; p0 += 8) {  // loads of eight parts in flight
        uint32_t x[8], y[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int p = min(p0 + q, parts - 1);
          const uint32_t* h = peer(hist(p & (H - 1)), p >> shift_H());
          const bool read = on && d <= last && p0 + q < parts;
          x[q] = read ? h[d] : 0u;
          y[q] = MASS && read ? h[kHist + d] : 0u;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) v += MASS ? (static_cast<uint64_t>(x[q]) << 14) + y[q] : x[q];
      }
      if (MASS) {
        v = v ? mass(v, d) : 0;
        const uint64_t s = warp_sum_u(v);
        if (lane < C && s) atomicAdd(reinterpret_cast<unsigned long long*>(peer(&S.Z, lane)), s);
      }
      const float f = static_cast<float>(v);
      if (on)
        for (int r = 0; r < C; ++r) peer(S.total, r)[d] = f;
    }
    sync_all();
  }

  // Bins -> the band between the first bin where the cut may lie and the first
  // where it must: where S.total's sum reaches `goal`, of masses good to 2^-18
  // (counts: exactly).  S.before: the count before the band.  False if the set
  // ends before.
  template <bool MASS>
  __device__ bool find_bins(float goal, Band& b) {
    constexpr int per = 4;
    const int b0 = threadIdx.x * per;
    float v[per] = {0.f, 0.f, 0.f, 0.f};
    if (b0 < kBins) {
      const float4 x = *reinterpret_cast<const float4*>(S.total + b0);
      v[0] = x.x;
      v[1] = x.y;
      v[2] = x.z;
      v[3] = x.w;
    }
    float all;
    float run = block_scan((v[0] + v[1]) + (v[2] + v[3]), S.fscratch, all);
    if (!MASS && all < goal) return false;
    constexpr float over = MASS ? 1.f + 0x1p-18f : 1.f, under = MASS ? 1.f - 0x1p-18f : 1.f;
    if (!MASS && run < goal) {  // counts are exact: one bin holds the cut
#pragma unroll
      for (int q = 0; q < per; ++q) {
        const float before = run;
        run += v[q];
        if (run >= goal && before < goal) {
          S.lo = S.hi = b0 + q;
          S.before = static_cast<int32_t>(before);
        }
      }
    }
    if (MASS) {
      // (The smallest of all such bins, not the one where a sum passes the goal: one
      // thread's sum and the next one's start differ by roundings.)
      int lo_bin = INT_MAX, hi_bin = INT_MAX;
#pragma unroll
      for (int q = 0; q < per; ++q) {
        run += v[q];
        if (v[q] > 0.f && run * over >= goal) lo_bin = min(lo_bin, b0 + q);
        if (v[q] > 0.f && run * under >= goal) hi_bin = min(hi_bin, b0 + q);
      }
      lo_bin = __reduce_min_sync(0xffffffffu, lo_bin);
      hi_bin = __reduce_min_sync(0xffffffffu, hi_bin);
      if (lane == 0 && lo_bin < INT_MAX) atomicMin(&S.lo, lo_bin);
      if (lane == 0 && hi_bin < INT_MAX) atomicMin(&S.hi, hi_bin);
    }
    __syncthreads();
    const int hi = min(S.hi, kBins - 1);
    set_band(b, min(S.lo, hi), hi);
    return true;
  }

  // Collects a superset of the set's k first tokens: the k-th largest of the
  // threads' own maxima (`mine`, two each) is a bound for the k-th largest
  // logit, so a histogram of those takes the place of one of every logit.
  // False where that names no band, or one too full to collect.
  __device__ bool collect_top(int k, const float (&mine)[2], Band& b) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (mine[u] >= zc) atomicAdd(&hist(sub)[max(0, sc.template bin<CLAMP>(mine[u]))], 1u);
    __syncthreads();
    merge<false>(kBins);
    if (!find_bins<false>(static_cast<float>(k), b)) return false;
    b.lo = 0;
    b.ehi = pos_inf();
    __syncthreads();  // (the histogram's place is the list's now)
    collect(b);
    return collected() <= kCap;
  }

  __device__ void set_band(Band& b, int lo, int hi) const {
    b.by_key = false;
    b.lo = lo;
    b.hi = hi;
    b.elo = hi >= kBins - 1 ? kNegMax : sc.edge(hi, -1);
    b.ehi = sc.edge(lo, 1);
  }

  // Collects the band's tokens, a list in each CTA; every CTA gets each CTA's
  // numbers: tokens above the band and in it, and per part S.mine (its weight in
  // bins before the band) with what tokens above the band but in its bins add.
  // Ends with a cluster barrier.
  __device__ void collect(const Band& b) {
    if (!b.by_key) {
      collect_bins(b);
      if (collected() <= kCap) return;
      sync_all();  // (everyone has read the counts)
      if (threadIdx.x == 0) S.above = S.ncollect = 0;
      __syncthreads();
    }
    collect_exact(b);
  }

  // ... for a band of bins: every token of the bins' range first, with the
  // test by bin after the pass, on the list.  Above kCap tokens in a CTA the
  // numbers are not complete.
  __device__ void collect_bins(const Band& b) {
    constexpr int VW = Elem<DT>::VW, G = 2;
    using Vec = typename Elem<DT>::Vec;
    uint32_t* raw = reinterpret_cast<uint32_t*>(list());
    int above = 0;
    sl.groups([&](const Vec(&x)[G], int j0) {
      unsigned zone = 0;  // a bit for each logit
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (DT == 0 && !(vec_max<DT>(x[g], neg_inf()) >= b.elo)) continue;
        float z[VW];
        Elem<DT>::unpack(x[g], z);
#pragma unroll
        for (int k = 0; k < VW; ++k) {
          above += z[k] >= b.ehi;
          if (z[k] >= b.elo && z[k] < b.ehi) zone |= 1u << (g * VW + k);
        }
      }
      if (!zone) return;
      int pos = atomicAdd(&S.ncollect, __popc(zone));
      const int i0 = sl.index(j0);
      while (zone) {  // (few; their logits are read again below, all at a time)
        const int bit = __ffs(zone) - 1;
        zone &= zone - 1;
        if (pos < kCap) raw[pos++] = i0 + 32 * VW * (bit / VW) + bit % VW;
      }
    });
    above = __reduce_add_sync(0xffffffffu, above);
    if (lane == 0 && above) atomicAdd(&S.above, above);
    if (threadIdx.x == 0) S.kept = 0;
    __syncthreads();
    const int n = min(S.ncollect, kCap);
    for (int i = threadIdx.x; i < n; i += kRowThreads) {
      const int idx = static_cast<int>(raw[i]);
      const float z = sl.logit(idx);
      if (!in_set(z, idx)) continue;
      const int pl = place(z, b);
      if (pl == 0) atomicAdd(&S.above, 1);
      else if (pl == 1) own_list()[atomicAdd(&S.kept, 1)] = token_key(z, idx);
    }
    __syncthreads();
    if (threadIdx.x < static_cast<unsigned>(C)) {
      const int r = threadIdx.x;
      peer(S.xabove, r)[rank] = S.above;
      peer(S.xcount, r)[rank] = S.ncollect > kCap ? kCap + 1 : S.kept;
#pragma unroll
      for (int h = 0; h < kMaxH; ++h)
        if (h < H) peer(S.xmass, r)[rank * H + h] = S.mine[h];
    }
    sync_all();
  }

  // ... for any band, the numbers complete whatever is collected.
  __device__ void collect_exact(const Band& b) {
    constexpr int VW = Elem<DT>::VW, G = 2;  // a mask bit for each logit of two vectors
    using Vec = typename Elem<DT>::Vec;
    int above = 0, in_band = 0;
    uint64_t acc = 0;
    sl.groups([&](const Vec(&x)[G], int j0) {
      unsigned zone = 0;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (DT == 0 && !(vec_max<DT>(x[g], neg_inf()) >= b.elo)) continue;
        float z[VW];
        Elem<DT>::unpack(x[g], z);
#pragma unroll
        for (int k = 0; k < VW; ++k) {
          above += z[k] >= b.ehi;
          if (z[k] >= b.elo && z[k] < b.ehi) zone |= 1u << (g * VW + k);
        }
      }
      while (zone) {  // (few: read again rather than kept in registers by number)
        const int bit = __ffs(zone) - 1;
        const int j = j0 + 32 * (bit / VW);
        zone &= zone - 1;
        const float z = sl.at(j, bit % VW);
        const int i = sl.index(j) + bit % VW;
        if (!in_set(z, i)) continue;
        const int pl = place(z, b);
        if (pl == 0) {
          ++above;
          if (!CLAMP && b.by_key && sc.template bin<false>(z) >= b.lo) acc += weight(z);
        } else if (pl == 1) {
          ++in_band;
          const int pos = atomicAdd(&S.ncollect, 1);
          if (pos < kCap) {
            own_list()[pos] = token_key(z, i);
          } else {  // (too many: the range of all of them is wanted)
            atomicMin(&S.kmin, order_key(z));
            atomicMax(&S.kmax, order_key(z));
          }
        }
      }
    });
    above = __reduce_add_sync(0xffffffffu, above);
    in_band = __reduce_add_sync(0xffffffffu, in_band);
    if (lane == 0) {
      if (above) atomicAdd(&S.above, above);
      if (in_band) atomicAdd(&S.band[sub], in_band);
    }
    if (!CLAMP && __any_sync(0xffffffffu, acc != 0)) {
      acc = warp_sum_u(acc);
      if (lane == 0) atomicAdd(reinterpret_cast<unsigned long long*>(&S.mass[sub]), acc);
    }
    __syncthreads();
    if (threadIdx.x < static_cast<unsigned>(C)) {
      const int r = threadIdx.x;
      peer(S.xabove, r)[rank] = S.above;
      peer(S.xcount, r)[rank] = S.ncollect;
#pragma unroll
      for (int h = 0; h < kMaxH; ++h)
        if (h < H) {
          peer(S.xband, r)[rank * H + h] = S.band[h];
          peer(S.xmass, r)[rank * H + h] = S.mine[h] + S.mass[h];
        }
    }
    sync_all();
  }

  // Tokens in the band collected last.
  __device__ int collected() const {
    int n = 0;
    for (int r = 0; r < C; ++r) n += S.xcount[r];
    return n;
  }

  // Over the cluster: tokens above the band, their weight.
  __device__ void before_band(int& above, uint64_t& w) const {
    above = 0;
    w = 0;
    for (int r = 0; r < C; ++r) above += S.xabove[r];
    for (int p = 0; p < C * H; ++p) w += S.xmass[p];
  }

  // A band that is too full: the range of its keys, on every CTA.
  __device__ void key_range(Band& b) {
    const int n = min(S.ncollect, kCap);
    uint32_t lo = 0xffffffffu, hi = 0;
    for (int i = threadIdx.x; i < n; i += kRowThreads) {
      const uint32_t k = ~static_cast<uint32_t>(own_list()[i] >> 32);
      lo = min(lo, k);
      hi = max(hi, k);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
      atomicMin(&S.kmin, lo);
      atomicMax(&S.kmax, hi);
    }
    __syncthreads();
    push_all(S.xkmin, rank, C, S.kmin);
    push_all(S.xkmax, rank, C, S.kmax);
    sync_all();
    for (int r = 0; r < C; ++r) {
      lo = min(lo, S.xkmin[r]);
      hi = max(hi, S.xkmax[r]);
    }
    b.kmin = lo;
    b.kmax = hi;
  }

  // Narrows a band too full to collect: counts by key over [kmin, kmax] into
  // 1024 bins.  count: the cut is the goal-th token of the band; else the
  // mass `goal` into it.  Bounds on a bin's mass (a bin spans up to a thousandth of a
  // wide range of keys) may leave the cut among too many tokens: then b is the lower
  // half of those bins, and S.upper the upper half's largest key (else 0).
  __device__ void narrow(Band& b, bool count, uint64_t goal) {
    constexpr int bins = 2 * kRowThreads;
    const uint32_t kmin = b.kmin, kmax = b.kmax;
    int shift = 0;
    while (((kmax - kmin) >> shift) >= static_cast<uint32_t>(bins)) ++shift;
    clear();
    sl.each([&](float z, int i) {
      if (z >= b.elo && z < b.ehi && in_set(z, i) && place(z, b) == 1) {
        const uint32_t key = order_key(z);
        if (key >= kmin && key <= kmax) atomicAdd(&hist(sub)[(kmax - key) >> shift], 1u);
      }
    });
    __syncthreads();
    merge<false>(bins);
    const int b0 = threadIdx.x * 2;
    uint64_t hw[2], lw[2];
    for (int q = 0; q < 2; ++q) {
      const uint32_t n = static_cast<uint32_t>(S.total[b0 + q]);
      const uint32_t top = kmax - (static_cast<uint32_t>(b0 + q) << shift);
      const uint32_t span = (1u << shift) - 1;
      const uint32_t low = top - kmin < span ? kmin : top - span;
      hw[q] = n == 0 ? 0 : count ? n : n * (weight(key_value(top)) + 1);
      lw[q] = n == 0 ? 0 : count ? n : n * weight(key_value(low));
    }
    uint64_t all;
    uint64_t hi_run = block_scan(hw[0] + hw[1], S.scratch, all);
    uint64_t lo_run = block_scan(lw[0] + lw[1], S.scratch, all);
    const bool exact = count || shift == 0;
    int last = -1;
    for (int q = 0; q < 2; ++q) {
      hi_run += hw[q];
      lo_run += lw[q];
      if (hw[q] == 0) continue;
      last = b0 + q;
      if ((exact ? lo_run : hi_run + (hi_run >> 28)) >= goal) atomicMin(&S.lo, b0 + q);
      if ((exact ? lo_run : lo_run - (lo_run >> 28)) >= goal) atomicMin(&S.hi, b0 + q);
    }
    if (threadIdx.x == 0) S.iscratch[0] = -1;
    __syncthreads();
    if (last >= 0) atomicMax(&S.iscratch[0], last);
    __syncthreads();
    const int end = S.iscratch[0];
    const int hi = min(S.hi, end), lo = min(S.lo, hi);
    b.by_key = true;
    b.kmax = kmax - (static_cast<uint32_t>(lo) << shift);
    if (!CLAMP && !exact && lo < hi) {  // (top logits count: always exact)
      uint64_t tokens = 0;
      for (int q = 0; q < 2; ++q)
        if (b0 + q >= lo && b0 + q <= hi) tokens += static_cast<uint64_t>(S.total[b0 + q]);
      if (block_sum_u(tokens) > kCap) {
        if (threadIdx.x == 0) S.upper = b.kmax;
        b.kmax = kmax - (static_cast<uint32_t>(((lo + hi) >> 1) + 1) << shift);
      }
    }
    const uint32_t last_top = kmax - (static_cast<uint32_t>(hi) << shift);
    const uint32_t span = (1u << shift) - 1;
    b.kmin = last_top - kmin < span ? kmin : last_top - span;
    b.elo = key_value(b.kmin);
    __syncthreads();
  }

  // The band at min-p's threshold zt, which lies in its bins: no tokens in it,
  // those from zt on above it.
  __device__ void set_given(Band& b, float zt) const {
    b.by_key = true;
    b.elo = fminf(b.elo, zt);
    b.kmax = order_key(zt) - 1;
    b.kmin = 0xffffffffu;
  }
  // No cut but the set's own: every token of it above the band.
  __device__ void set_whole(Band& b) const {
    b.by_key = true;
    b.lo = b.hi = kBins;
    b.elo = zc;
    b.ehi = key_value(order_key(zc) + 1);
    b.kmax = 0;
    b.kmin = 0xffffffffu;
  }

  // Cuts the set at the goal-th token, where the mass `goal` is reached, or
  // (kGiven) at zt, starting from a band of bins, and sets zc, ic.  `fin`: the
  // last cut, whose sums give the token as well (min-p's threshold zt is then
  // part of it).
  __device__ void cut(Band b, CutKind kind, uint64_t goal, bool fin, float zt, const float* u) {
    for (int it = 0; it < 80; ++it) {  // (each two turns halve the band's keys; three are the usual most)
      if (fin && (CLAMP || S.upper == 0) && kind != kGiven && b.by_key && order_key(zt) > b.kmax) {  // min-p ends the kept tokens first
        set_given(b, zt);
        kind = kGiven;
      }
      collect(b);
      const int n = collected();
      int above;
      uint64_t w;
      before_band(above, w);
      if (!CLAMP && S.upper != 0) {  // which half the cut lies in, by the exact mass above the lower one
        if (w >= goal) {
          b.kmin = b.kmax + 1;
          b.kmax = S.upper;
          b.elo = key_value(b.kmin);
        }
        sync_all();  // (everyone has read the masses)
        clear();
        continue;
      }
      if (n <= kCap) {
        if (rank == 0) resolve(n, above, w, kind, goal, fin, zt, u);
        publish();
        break;
      }
      key_range(b);
      const float z = key_value(b.kmin);
      if (b.kmin == b.kmax) {
        if (rank == 0) resolve_tie(n, above, w, z, kind, goal, fin, zt, u);
        publish();
        find_tie(z);
        break;
      }
      const uint64_t before = kind == kByCount ? static_cast<uint64_t>(above) : w;
      narrow(b, kind == kByCount, goal > before ? goal - before : 0);
    }
    zc = S.dec.zc;
    ic = S.dec.ic;
  }

  // Rank 0: the n <= kCap collected tokens of all CTAs into list().
  __device__ void pull(int n) {
    for (int t = threadIdx.x; t < n; t += kRowThreads) {
      int r = 0, i = t;
      while (i >= S.xcount[r]) i -= S.xcount[r++];
      list()[t] = peer(work, r)[i];
    }
    __syncthreads();
  }

  // Sorts n <= kCap tokens through bins of their range of keys, a thread's each:
  // within a bin every token counts those before it.  bf16 logits have few
  // values in a band and many tokens of each: there a bin is a value and a
  // range of indices.  False (nothing done) where a bin is too full.
  __device__ bool sort_by_bins(uint64_t* a, int n) {
    uint32_t* count = reinterpret_cast<uint32_t*>(S.total);
    uint32_t lo = 0xffffffffu, hi = 0;
    constexpr int per = kCap / kRowThreads;
    uint64_t x[per];
#pragma unroll
    for (int q = 0; q < per; ++q) {
      const int i = threadIdx.x + q * kRowThreads;
      x[q] = i < n ? a[i] : ~0ull;
      if (i < n) {
        lo = min(lo, static_cast<uint32_t>(x[q] >> 32));
        hi = max(hi, static_cast<uint32_t>(x[q] >> 32));
      }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    __syncthreads();  // (S.total and the scratch are free)
    if (lane == 0) S.scratch[warp] = (static_cast<uint64_t>(lo) << 32) | hi;
    count[threadIdx.x] = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) {
      lo = min(lo, static_cast<uint32_t>(S.scratch[w] >> 32));
      hi = max(hi, static_cast<uint32_t>(S.scratch[w]));
    }
    const uint32_t values = ((hi - lo) >> 16) + 1;
    const bool by_value = DT == 0 && values <= kRowThreads;
    const int shift = by_value ? 16 : max(0, 32 - __clz(hi - lo) - 9);
    const uint32_t wide = by_value ? kRowThreads / values : 1;  // bins per value
    const uint32_t scale = wide * (0xffffffffu / static_cast<uint32_t>(V));
    auto bin = [&](uint64_t t) {
      const uint32_t v = (static_cast<uint32_t>(t >> 32) - lo) >> shift;
      return by_value ? v * wide + __umulhi(static_cast<uint32_t>(t), scale) : v;
    };
    int at[per];
#pragma unroll
    for (int q = 0; q < per; ++q)
      if (x[q] != ~0ull) at[q] = atomicAdd(&count[bin(x[q])], 1u);
    __syncthreads();
    const uint32_t mine = count[threadIdx.x];
    const bool full = __syncthreads_or(mine > 64);
    if (full) return false;
    uint32_t all;
    const uint32_t start = block_scan(mine, reinterpret_cast<uint32_t*>(S.iscratch), all);
    count[threadIdx.x] = start << 16 | mine;
    __syncthreads();
    // binned into place, then counted within the bin
#pragma unroll
    for (int q = 0; q < per; ++q)
      if (x[q] != ~0ull) a[(count[bin(x[q])] >> 16) + at[q]] = x[q];
    __syncthreads();
#pragma unroll
    for (int q = 0; q < per; ++q)
      if (x[q] != ~0ull) {
        const uint32_t c = count[bin(x[q])];
        at[q] = c >> 16;
        for (uint32_t j = c >> 16; j < (c >> 16) + (c & 0xffffu); ++j) at[q] += a[j] < x[q];
      }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < per; ++q)
      if (x[q] != ~0ull) a[at[q]] = x[q];
    __syncthreads();
    return true;
  }

  // Sorts n <= kCap tokens.  By bins in the place of counts, 32 tokens of 4 rows of
  // 32000 take 15 % longer.  By exchanges in the place of bins (as where a bin is too
  // full), the 256 largest of 2048 x 152064 bf16 20 %, a draw from 2304 x 152064 fp32
  // 15 %.
  __device__ void sort(uint64_t* a, int n) {
    int P = 16;
    while (P < n) P <<= 1;
    if (P <= kRowThreads / 2) {  // few: G threads count the tokens before each
      const int G = kRowThreads / P, i = threadIdx.x / G, sub = threadIdx.x % G;
      const uint64_t x = i < n ? a[i] : 0;
      int before = 0;
      for (int j = sub; j < n; j += G) before += a[j] < x;
      for (int o = G / 2; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
      __syncthreads();
      if (sub == 0 && i < n) a[before] = x;
      __syncthreads();
      return;
    }
    if (sort_by_bins(a, n)) return;
    if (n > 2 * kRowThreads) {  // equal logits, most likely: every token counts all before it
      constexpr int per = kCap / kRowThreads;
      uint64_t x[per];
      int at[per] = {};
#pragma unroll
      for (int q = 0; q < per; ++q) x[q] = threadIdx.x + q * kRowThreads < n ? a[threadIdx.x + q * kRowThreads] : ~0ull;
      for (int j = 0; j < n; ++j)
#pragma unroll
        for (int q = 0; q < per; ++q) at[q] += a[j] < x[q];
      __syncthreads();
#pragma unroll
      for (int q = 0; q < per; ++q)
        if (x[q] != ~0ull) a[at[q]] = x[q];
      __syncthreads();
      return;
    }
    // two tokens a thread (places 2 t and 2 t + 1), steps below 64 within a warp
    uint64_t p = ~0ull, q = ~0ull;
    const int i = 2 * threadIdx.x;
    if (i < n) p = a[i];
    if (i + 1 < n) q = a[i + 1];
    for (int size = 2; size <= P; size <<= 1) {
      const bool up = (i & size) == 0;
      for (int step = size >> 1; step > 0; step >>= 1) {
        if (step == 1) {
          if ((p > q) == up) {
            const uint64_t t = p;
            p = q;
            q = t;
          }
          continue;
        }
        uint64_t x, y;
        if (step < 64) {
          x = __shfl_xor_sync(0xffffffffu, p, step >> 1);
          y = __shfl_xor_sync(0xffffffffu, q, step >> 1);
        } else {
          __syncthreads();
          if (i < P) {
            a[i] = p;
            a[i + 1] = q;
          }
          __syncthreads();
          x = i < P ? a[i ^ step] : p;
          y = i < P ? a[(i + 1) ^ step] : q;
        }
        const bool lower = (i & step) == 0;
        if ((p > x) == (lower == up)) p = x;
        if ((q > y) == (lower == up)) q = y;
      }
    }
    __syncthreads();
    if (i < n) a[i] = p;
    if (i + 1 < n) a[i + 1] = q;
    __syncthreads();
  }

  // Rank 0, the band collected: where the cut falls in it.
  __device__ void resolve(int n, int above, uint64_t w, CutKind kind, uint64_t goal, bool fin, float zt, const float* u) {
    const bool count = kind == kByCount;
    if (threadIdx.x == 0) S.lo = n - 1;
    pull(n);
    sort(list(), n);
    constexpr int per = kCap / kRowThreads;
    const int i0 = threadIdx.x * per;
    uint64_t v[per], x = 0;
    float z[per];
#pragma unroll
    for (int q = 0; q < per; ++q) {
      z[q] = i0 + q < n ? token_logit(list()[i0 + q]) : 0.f;
      v[q] = i0 + q < n ? (count ? 1ull : weight(z[q])) : 0;
      x += v[q];
    }
    uint64_t all;
    uint64_t run = (count ? static_cast<uint64_t>(above) : w) + block_scan(x, S.scratch, all);
#pragma unroll
    for (int q = 0; q < per; ++q) {
      run += v[q];
      if (i0 + q < n && run >= goal) atomicMin(&S.lo, i0 + q);
      if (i0 + q < n && fin && z[q] < zt) atomicMin(&S.lo, i0 + q - 1);  // min-p ends the kept tokens
    }
    __syncthreads();
    const int nb = S.lo + 1;  // the band's tokens that the cut keeps
    if (kind == kGiven || nb == 0) {
      zc = zt;
      ic = INT_MAX;
    } else {
      zc = token_logit(list()[nb - 1]);
      ic = token_index(list()[nb - 1]);
    }
    if (threadIdx.x == 0) {
      S.dec.tie_part = -1;
      S.dec.zc = zc;
      S.dec.ic = ic;
      S.dec.kept = above + nb;
    }
    if (fin && u) finish(nb, 0, 0.f, *u);
  }

  // Rank 0, every token down to the k-th's bin collected (n of them): top-k,
  // top-p, min-p and the draw on the sorted list.
  __device__ void resolve_top(int n, int k, float tp, float zt, const float* u) {
    pull(n);
    sort(list(), n);
    const int m = min(k, n);
    constexpr int per = kCap / kRowThreads;
    const int i0 = threadIdx.x * per;
    uint64_t v[per], x = 0;
#pragma unroll
    for (int q = 0; q < per; ++q) {
      v[q] = i0 + q < m ? weight(token_logit(list()[i0 + q])) : 0;
      x += v[q];
    }
    uint64_t all;
    uint64_t run = block_scan(x, S.scratch, all);
    uint64_t goal = tp < 1.f ? fraction(tp, all) + 1 : all;
    goal -= goal >> kSlack;
    if (threadIdx.x == 0) S.lo = m - 1;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < per; ++q) {
      run += v[q];
      if (i0 + q < m && tp < 1.f && run >= goal) atomicMin(&S.lo, i0 + q);
      if (i0 + q < m && i0 + q > 0 && token_logit(list()[i0 + q]) < zt) atomicMin(&S.lo, i0 + q - 1);
    }
    __syncthreads();
    const int nk = S.lo + 1;
    zc = token_logit(list()[nk - 1]);
    ic = token_index(list()[nk - 1]);
    if (threadIdx.x == 0) {
      S.dec.tie_part = -1;
      S.dec.zc = zc;
      S.dec.ic = ic;
      S.dec.kept = nk;
    }
    if (!u) return;
    if (nk > kRowThreads / 2) {
      finish(nk, 0, 0.f, *u);
      return;
    }
    // The draw: G threads add up the weights of lower index for each.  (In place
    // of a part's sums and a pass over it: 50 tokens of a row of 32000 19 us, 25.)
    uint64_t* wt = reinterpret_cast<uint64_t*>(S.total);
#pragma unroll
    for (int q = 0; q < per; ++q) {
      if (i0 + q < nk) wt[i0 + q] = v[q];
      else v[q] = 0;
    }
    x = 0;
#pragma unroll
    for (int q = 0; q < per; ++q) x += v[q];
    const uint64_t W = block_sum_u(x);
    const bool fell = !(*u < 1.f);
    uint64_t t = *u > 0.f && !fell ? fraction(*u, W) : 0;
    t += t >> kSlack;
    int P = 16;
    while (P < nk) P <<= 1;
    const int G = kRowThreads / P, i = threadIdx.x / G, sub = threadIdx.x % G;
    const int idx = i < nk ? token_index(list()[i]) : -1;
    uint64_t before = 0;
    bool last = true;
    for (int j = sub; j < nk; j += G) {
      const int other = token_index(list()[j]);
      before += other < idx ? wt[j] : 0;
      last = last && other <= idx;
    }
    for (int o = G / 2; o > 0; o >>= 1) {
      before += __shfl_xor_sync(0xffffffffu, before, o);
      last = __shfl_xor_sync(0xffffffffu, last, o) && last;
    }
    if (sub == 0 && i < nk && (fell ? last : before <= t && (t < before + wt[i] || last))) {
      S.dec.part = -1;
      S.dec.token = idx;
      S.dec.z = token_logit(list()[i]);
      S.dec.W = W;
      S.dec.fallback = fell;
    }
    __syncthreads();
  }

  // Rank 0, a band of n > kCap equal logits: how many of them are kept, and
  // which part holds the last one.
  __device__ void resolve_tie(int n, int above, uint64_t w, float z, CutKind kind, uint64_t goal, bool fin, float zt,
                              const float* u) {
    const bool count = kind == kByCount;
    const uint64_t before = count ? static_cast<uint64_t>(above) : w, one = count ? 1 : weight(z);
    const uint64_t left_over = goal > before ? goal - before : 0;
    int nb = static_cast<int>(min(max((left_over + one - 1) / one, uint64_t(1)), static_cast<uint64_t>(n)));
    if (fin && z < zt) nb = 0;
    if (threadIdx.x == 0) {
      S.dec.tie_part = -1;
      S.dec.zc = nb > 0 ? z : zt;
      S.dec.ic = INT_MAX;
      S.dec.kept = above + nb;
      int left = nb;
      for (int p = 0; p < C * H && left > 0; ++p) {
        if (S.xband[p] >= left) {
          S.dec.tie_part = p;
          S.dec.tie_rank = left - 1;
          break;
        }
        left -= S.xband[p];
      }
    }
    __syncthreads();
    if (fin && u) finish(0, nb, z, *u);
  }

  // The index of the tie_rank-th logit equal to z in part tie_part, to every CTA.
  __device__ void find_tie(float z) {
    if (S.dec.tie_part >= 0 && S.dec.tie_part >> shift_H() == rank) {
      int mine = 0;
      sl.each([&](float x, int i) { mine += x == z && in_set(x, i); });
      mine = __reduce_add_sync(0xffffffffu, mine);
      int left = S.dec.tie_rank;
      __syncthreads();
      if (lane == 0) S.iscratch[warp] = mine;
      __syncthreads();
      const bool here_part = (S.dec.tie_part & (H - 1)) == sub;
      for (int w = sub * (kRowWarps >> shift_H()); w < warp; ++w) left -= S.iscratch[w];
      if (here_part && left >= 0 && left < mine) {  // this warp's segment
        for (int j0 = 0; j0 < sl.nv && left >= 0; j0 += 32) {
          const int j = j0 + lane, i0 = sl.index(j);
          float x[Elem<DT>::VW];
          int here = 0;
          if (j < sl.nv) {
            Elem<DT>::unpack(sl.vec(j), x);
#pragma unroll
            for (int q = 0; q < Elem<DT>::VW; ++q) here += x[q] == z && in_set(x[q], i0 + q);
          }
          int inc = here;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
          }
          int at = left - (inc - here);
          if (here > 0 && at >= 0 && at < here) {
#pragma unroll
            for (int q = 0; q < Elem<DT>::VW; ++q)
              if (x[q] == z && in_set(x[q], i0 + q) && at-- == 0)
                for (int r = 0; r < C; ++r) peer(&S.dec, r)->ic = i0 + q;
          }
          left -= __shfl_sync(0xffffffffu, inc, 31);
        }
      }
    }
    sync_all();
  }

  // a / b for 0 <= a < 2^24.
  __device__ __forceinline__ static int quotient(int a, int b) {
    int q = static_cast<int>(__fdividef(static_cast<float>(a), static_cast<float>(b)));
    q -= q * b > a;
    return q + ((q + 1) * b <= a);
  }

  // Rank 0: total weight of the kept tokens, and the part where the running sum
  // in index order passes u times it.  Kept: the parts' weights above the band,
  // those of the first n_list tokens of list(), and the first nt logits equal
  // to z.
  __device__ void finish(int n_list, int nt, float z, float u) {
    if (threadIdx.x < 3 * kMaxParts) S.fix32[threadIdx.x / kMaxParts][threadIdx.x % kMaxParts] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n_list; i += kRowThreads) {
      const uint64_t k = list()[i], w = weight(token_logit(k));
      const int vec = token_index(k) / Elem<DT>::VW, cta = quotient(vec, split.svec);
      const int part = cta * H + ((quotient(vec - cta * split.svec, split.gvec) << shift_H()) / kRowWarps);
      atomicAdd(&S.fix32[0][part], static_cast<uint32_t>(w) & 0x7fffu);
      atomicAdd(&S.fix32[1][part], static_cast<uint32_t>(w >> 15) & 0x7fffu);
      atomicAdd(&S.fix32[2][part], static_cast<uint32_t>(w >> 30));
    }
    __syncthreads();
    if (threadIdx.x < 32) {  // a lane per part
      const bool on = lane < C * H;
      uint64_t x = 0;
      int ties = on && nt > 0 ? S.xband[lane] : 0;
      if (on)
        x = S.xmass[lane] + S.fix32[0][lane] + (static_cast<uint64_t>(S.fix32[1][lane]) << 15) +
            (static_cast<uint64_t>(S.fix32[2][lane]) << 30);
      if (nt > 0) {
        int inc = ties;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        ties = max(0, min(ties, nt - (inc - ties)));
        x += weight(z) * static_cast<uint64_t>(ties);
      }
      uint64_t inc = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      const uint64_t W = __shfl_sync(0xffffffffu, inc, 31);
      const bool fell = !(u < 1.f);
      // (whole numbers: a sum exceeds u W exactly if it exceeds its floor)
      uint64_t t = u > 0.f && !fell ? fraction(u, W) : 0;
      t += t >> kSlack;
      const unsigned over = __ballot_sync(0xffffffffu, x > 0 && !fell && inc > t);
      const unsigned some = __ballot_sync(0xffffffffu, x > 0);
      const int who = over ? __ffs(over) - 1 : 31 - __clz(some);
      if (lane == who) {
        S.dec.part = lane;
        S.dec.rem = fell ? ~0ull : t - (inc - x);
        S.dec.W = W;
        S.dec.fallback = fell;
      }
    }
  }

  __device__ void publish() {  // rank 0's decision to every CTA
    __syncthreads();
    if (rank == 0) {
      const Decision d = S.dec;
      if (static_cast<int>(threadIdx.x) < C && threadIdx.x > 0) *peer(&S.dec, static_cast<int>(threadIdx.x)) = d;
    }
    sync_all();
  }

  // The CTA that the token's part `p` lies in: the first kept token whose
  // running sum from the part's start exceeds `rem`, or its last one.  Every
  // warp takes a piece of the part.
  __device__ void draw(const void* row, int p, uint64_t rem, uint64_t W, int32_t* token, float* prob) {
    constexpr int VW = Elem<DT>::VW;
    const int per = kRowWarps >> shift_H();  // segments of the part
    Slice piece =
        sl.piece(smem, S.bars, split, row, rank, (p & (H - 1)) * per + (warp >> shift_H()), warp & (H - 1), H);
    // sums of up to 32 blocks of the warp's piece, a lane's each
    const int per_block = (piece.nv + 32 * kStage - 1) / (32 * kStage) * kStage;
    uint64_t block = 0;
    piece.groups([&](const typename Elem<DT>::Vec(&x)[2], int j) {
      uint64_t sum = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float z[VW];
        Elem<DT>::unpack(x[h], z);
        const int i0 = piece.index(j + 32 * h);
#pragma unroll
        for (int q = 0; q < VW; ++q)
          if (in_set(z[q], i0 + q)) sum += weight(z[q]);
      }
      sum = warp_sum_u(sum);
      if (lane == (j - lane) / per_block) block += sum;
    });
    uint64_t inc = block;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const uint64_t mine = __shfl_sync(0xffffffffu, inc, 31);
    __syncthreads();
    if (lane == 0) S.scratch[warp] = mine;
    __syncthreads();
    uint64_t run = 0;
    bool later = false;  // a later warp holds kept tokens
    for (int w = 0; w < kRowWarps; ++w) {
      if (w < warp) run += S.scratch[w];
      later |= w > warp && S.scratch[w] > 0;
    }
    if (mine == 0 || run > rem || (run + mine <= rem && later)) return;
    // this warp's piece: the block, or else the last that holds kept tokens
    const unsigned past = __ballot_sync(0xffffffffu, block > 0 && run + inc > rem);
    const int at = past ? __ffs(past) - 1 : 31 - __clz(__ballot_sync(0xffffffffu, block > 0));
    run += __shfl_sync(0xffffffffu, inc - block, at);
    int last = -1, found = -1;
    float lastz = 0.f, tz = 0.f;
    for (int j0 = at * per_block; j0 < min(piece.nv, (at + 1) * per_block); j0 += 32) {
      const int j = j0 + lane;
      const int i0 = piece.index(j);
      float z[VW];
      uint64_t w[VW], x = 0;
      if (j < piece.nv) Elem<DT>::unpack(piece.vec(j), z);
#pragma unroll
      for (int q = 0; q < VW; ++q) {
        const bool in = j < piece.nv && in_set(z[q], i0 + q);
        w[q] = in ? weight(z[q]) : 0;
        x += w[q];
        if (in) {
          last = i0 + q;
          lastz = z[q];
        }
      }
      uint64_t upto = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const unsigned over = __ballot_sync(0xffffffffu, x > 0 && run + upto > rem);
      if (over) {
        const int who = __ffs(over) - 1;
        if (lane == who) {
          uint64_t y = run + upto;
#pragma unroll
          for (int q = VW - 1; q >= 0; --q) {  // the first whose sum passes: from the end
            if (w[q] > 0 && y > rem) {
              found = i0 + q;
              tz = z[q];
            }
            y -= w[q];
          }
        }
        found = __shfl_sync(0xffffffffu, found, who);
        tz = __shfl_sync(0xffffffffu, tz, who);
        break;
      }
      run += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (found < 0) {  // the piece's last kept token
      const int most = __reduce_max_sync(0xffffffffu, last);
      const int who = __ffs(__ballot_sync(0xffffffffu, last == most)) - 1;
      found = most;
      tz = __shfl_sync(0xffffffffu, lastz, who);
    }
    if (lane == 0) {
      *token = found;
      if (prob) *prob = share(tz, W);
    }
  }
};

// One row per cluster: the cut, the token, the filtered logits.
// Many rows are bound by issue slots and shared atomics: 2304 x 152064 fp32 top-p
// 0.93 ms (1401 MB, 1.51 TB/s), of a row's time a third in the pass for the
// masses (25 operations and two atomics a logit), a fifth in the band's
// collection, the rest in the merge, the sorted list and the draw.  320 x 128256
// bf16 filtered 112 to 118 us by the rules drawn (164 MB).  Few rows are bound by the chain of these steps,
// 1 to 3 us each: one row of 32000 with top-k 16 us, 32 x 128256 bf16 mixed 34.
template <int DT>
__global__ void __launch_bounds__(kRowThreads, 2) sample_filter_kernel(const __grid_constant__ FilterParams P) {
  using E = Elem<DT>;
  extern __shared__ __align__(128) char smem[];
  __shared__ __align__(16) FilterShared S;
  const int C = P.sp.C, V = P.sp.V;
  const int64_t row = blockIdx.x / C;
  const int64_t b = row / P.R;
  cluster_arrive();  // waited for before the first remote write
  const char* zrow = reinterpret_cast<const char*>(P.z) + (b * P.bs + (row - b * P.R) * P.rs) * E::ES;
  FilterRow<DT, false> F(S, P.sp, smem, zrow);
  const int rank = F.rank, lane = F.lane, warp = F.warp;
  F.sl.load();
  if (threadIdx.x < kGrid) {
    S.tab[threadIdx.x] = P.tab.e[threadIdx.x];
    S.tab32[threadIdx.x] = static_cast<uint32_t>((P.tab.e[threadIdx.x] + 0x80000000u) >> 32);
  }
  if (threadIdx.x == 0) S.bad = 0;
  if (threadIdx.x < kMaxH) S.mine[threadIdx.x] = 0;
  const float T = P.temp[b];
  const int k = P.top_k ? P.top_k[b] : 0;
  const float tp = P.top_p ? P.top_p[b] : 1.f;
  const float mp = P.min_p ? P.min_p[b] : 0.f;
  const float* u = P.u ? P.u + row : nullptr;
  int bad = 0;
  if (!(T >= 0.f) || T > 3.4e38f) bad |= kBadTemp;
  if (k < 0 || !(tp >= 0.f && tp <= 1.f) || !(mp >= 0.f && mp <= 1.f)) bad |= kBadFilter;
  // Thresholds below the maximum in fp64, by one thread while the copies run.
  const float Tc = fmaxf(T, 1e-30f);
  double tf = 0, tm = 0;
  if (threadIdx.x == 0) {
    const double lnf = -kWindow * 0.69314718055994530942;
    tf = static_cast<double>(Tc) * lnf;
    tm = mp > 0.f ? static_cast<double>(Tc) * fmax(log(static_cast<double>(mp)), lnf) : tf;
  }
  __syncthreads();
  cluster_wait();
  // Streamed rows without top-k: masses and maximum in one pass.
  bool guessed = P.sp.rvec < P.sp.gvec && bad == 0 && T > 0.f && (k == 0 || k >= V) && (tp < 1.f || u);
  float own[2], wm;
  if (guessed) {
    F.sc.set_factor(Tc);
    const float m0 = F.guess_max();
    guessed = fabsf(m0) * F.sc.chi < 16000.f;  // (false for infinities and NaN)
    if (guessed) {
      F.sc.set_max(m0);
      if (threadIdx.x == 0) S.zf = __double2float_ru(static_cast<double>(m0) + tf);
      F.off = kHead;
      F.clear();  // (a barrier)
      wm = F.max_and_masses(S.zf);
    }
  }
  if (!guessed) wm = F.sl.warp_max(own);
  if (F.sl.late) atomicOr(&S.bad, kTimeout);
  const float mc = block_max_nan(wm, S.fscratch);
  push_all(S.xmax, rank, C, mc);
  push_all(S.xbad, rank, C, S.bad);
  F.sync_all();
  float m = neg_inf();
  for (int r = 0; r < C; ++r) {
    m = max_nan(m, S.xmax[r]);
    bad |= S.xbad[r];
  }
  if (!(m > neg_inf() && m < pos_inf())) bad |= kNonFinite;

  F.zc = pos_inf();  // (nothing kept)
  F.ic = -1;
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
    F.sync_all();
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
    F.sc.set_factor(Tc);
    const int guess = F.sc.gm;
    F.sc.set_max(m);
    if (guessed) {
      // (A maximum that is shifted first lies on another grid: no place of it is
      // comparable with the guess.)
      F.off += guess - F.sc.gm;
      guessed = F.sc.shift == 0.f && F.off >= 0 && F.off <= kHead;
      if (!guessed) F.off = 0;
    }
    if (threadIdx.x == 0) {
      S.zf = __double2float_ru(static_cast<double>(m) + tf);
      S.zt = fmaxf(S.zf, __double2float_ru(static_cast<double>(m) + tm));
    }
    if (guessed) __syncthreads();
    else F.clear();  // (a barrier)
    const float zf = S.zf, zt = S.zt;
    F.zc = zf;
    F.ic = INT_MAX;
    const bool use_k = k > 0 && k < V, use_p = tp < 1.f;
    Band band;
    bool done = false;
    if (use_k && kFewTop * k <= 2 * C * kRowThreads) {
      if (F.collect_top(k, own, band)) {
        if (rank == 0) F.resolve_top(F.collected(), k, tp, zt, u);
        F.publish();
        F.zc = S.dec.zc;
        F.ic = S.dec.ic;
        done = true;
      } else {
        F.clear();
      }
    }
    if (use_k && !done) {
      F.sl.each([&](float z, int) {
        if (z >= zf) atomicAdd(&F.hist(F.sub)[F.sc.template bin<false>(z)], 1u);
      });
      __syncthreads();
      F.template merge<false>(kBins);
      if (F.template find_bins<false>(static_cast<float>(k), band)) {
        const int upto = S.before + static_cast<int>(S.total[band.hi]);
        __syncthreads();
        if (upto <= kCap) {  // few enough to collect: the rest is done on the list
          band.lo = 0;
          band.ehi = pos_inf();
          F.collect(band);
          if (rank == 0) F.resolve_top(F.collected(), k, tp, zt, u);
          F.publish();
          F.zc = S.dec.zc;
          F.ic = S.dec.ic;
          done = true;
        } else {
          done = !use_p && !u;
          CutKind kind = kByCount;
          if (done && zt > zf) {
            const int dt = F.sc.template bin<false>(zt);
            if (dt < band.lo) {  // min-p ends the kept tokens first
              F.set_band(band, dt, dt);
              F.set_given(band, zt);
              kind = kGiven;
            }
          }
          F.cut(band, kind, k, done, zt, u);
        }
      }
      if (!done) F.clear();
    }
    if (!done) {
      uint64_t goal = 0;
      CutKind kind = kGiven;
      int last = 0;  // the last bin that counts
      if (use_p || u) {
        const float cut = F.zc;
        const bool whole = F.ic == INT_MAX;
        const uint32_t to = F.base();
        const int top = F.most();
        // (Below a guessed maximum the last bin holds tokens under the floor too.  All of
        // it is left out, at most 2^-47.9 for each of its kept ones: a part is drawn from
        // only if it holds kept tokens.)
        last = F.sc.template bin<false>(zf) - (guessed ? 1 : 0);
        if (guessed) {
        } else if (whole) {
          F.sl.each([&](float z, int) {
            F.template add_mass<true>(to, top, z, cut, true);
          });
        } else {
          F.sl.each([&](float z, int i) {
            F.template add_mass<true>(to, top, z, cut, F.in_set(z, i));
          });
        }
        __syncthreads();
        F.template merge<true>(kBins, last);
        if (use_p) {
          goal = fraction(tp, S.Z) + 1;
          goal -= goal >> kSlack;
          F.template find_bins<true>(static_cast<float>(goal), band);
          kind = kByMass;
        }
      }
      if (zt > F.zc) {  // min-p's threshold, where it ends the kept tokens
        const int dt = F.sc.template bin<false>(zt);
        if (kind == kGiven || dt < band.lo) {
          F.set_band(band, dt, dt);
          F.set_given(band, zt);
          kind = kGiven;
        }
      } else if (kind == kGiven) {
        F.set_whole(band);
      }
      if (use_p || u) {  // the parts' weights in the bins before the band
        // (a part's bins shared by its own warps)
        uint64_t x = 0;
        const int width = kRowThreads / P.sp.H;
        const uint32_t* hist = F.hist(F.sub);
        for (int d = threadIdx.x % width; d < min(band.lo, last + 1); d += width) {
          const uint64_t v = (static_cast<uint64_t>(hist[d]) << 14) + hist[kHist + d];
          if (v) x += max(F.mass(v, d), uint64_t(1));
        }
        x = warp_sum_u(x);
        if (lane == 0) S.scratch[warp] = x;
        __syncthreads();  // (and the histogram's place is the list's now)
        if (static_cast<int>(threadIdx.x) < P.sp.H) {
          const int per = kRowWarps / P.sp.H;
          x = 0;
          for (int w = 0; w < per; ++w) x += S.scratch[threadIdx.x * per + w];
          S.mine[threadIdx.x] = x;
        }
      }
      // (without a cut of its own, the set's)
      const float zg = kind == kGiven ? fmaxf(zt, F.zc) : zt;
      if (kind == kGiven && zt <= F.zc) {
        F.collect(band);
        if (rank == 0) {
          int above;
          uint64_t w;
          F.before_band(above, w);
          if (threadIdx.x == 0) {
            S.dec.zc = F.zc;
            S.dec.ic = F.ic;
            S.dec.kept = above;
          }
          if (u) F.finish(0, 0, 0.f, *u);
        }
        F.publish();
      } else {
        F.cut(band, kind, goal, true, zg, u);
      }
    }
    if (rank == 0 && threadIdx.x == 0) {
      if (P.kept) P.kept[row] = S.dec.kept;
      if (P.status) P.status[row] = (u && S.dec.fallback) ? kFallback : 0;
      if (u && S.dec.part < 0) {
        P.tokens[row] = S.dec.token;
        if (P.prob) P.prob[row] = F.share(S.dec.z, S.dec.W);
      }
    }
    if (u && S.dec.part >= 0 && S.dec.part >> F.shift_H() == rank)
      F.draw(zrow, S.dec.part, S.dec.rem, S.dec.W, P.tokens + row, P.prob ? P.prob + row : nullptr);
  }

  if (P.out) {
    char* orow = reinterpret_cast<char*>(P.out) + (b * P.obs + (row - b * P.R) * P.ors) * E::ES;
    F.sl.groups([&](const typename E::Vec(&x)[2], int j) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i0 = F.sl.index(j + 32 * h);
        float z[E::VW];
        E::unpack(x[h], z);
#pragma unroll
        for (int q = 0; q < E::VW; ++q) z[q] = F.in_set(z[q], i0 + q) ? z[q] : neg_inf();
        store_warp<DT>(orow, i0, V, j + 32 * h < F.sl.nv, pack_vec<DT>(z));
      }
    });
  }
}

// One row per cluster: the k largest logits, in order, and the log-sum-exp.
// 256 of 2048 x 152064 bf16 234 us (623 MB, 2.7 TB/s): a row's collection and
// sort follow its pass for maximum and sum, and the other CTA on the SM covers
// only part of them.  32 of 4 x 32000 fp32 11 us, 100 of 333 x 50257 fp32 42.
template <int DT>
__global__ void __launch_bounds__(kRowThreads, 2) top_logits_kernel(const __grid_constant__ TopParams P) {
  using E = Elem<DT>;
  extern __shared__ __align__(128) char smem[];
  __shared__ __align__(16) FilterShared S;
  const int C = P.sp.C, k = P.k;
  const int64_t row = blockIdx.x / C;
  cluster_arrive();
  FilterRow<DT, true> F(S, P.sp, smem, reinterpret_cast<const char*>(P.z) + row * P.rs * E::ES);
  const int rank = F.rank, lane = F.lane, warp = F.warp;
  F.sl.load();
  if (threadIdx.x == 0) S.bad = 0;
  if (threadIdx.x < kMaxH) S.mine[threadIdx.x] = 0;
  F.clear();  // (a barrier)
  float own[2];
  RunningSum rs;  // (the log-sum-exp's share, in the same pass)
  const float wm = F.sl.warp_max(own, &rs, P.c);
  if (F.sl.late) atomicOr(&S.bad, kTimeout);
  const float mc = block_max_nan(wm, S.fscratch);
  cluster_wait();
  push_all(S.xmax, rank, C, mc);
  push_all(S.xbad, rank, C, S.bad);
  F.sync_all();
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
  float s = rs.at(m, P.c);
  s = warp_sum_f(s);
  if (lane == 0) S.fscratch[warp] = s;
  __syncthreads();
  s = 0.f;
#pragma unroll
  for (int w = 0; w < kRowWarps; ++w) s += S.fscratch[w];
  push_all(S.xexp, rank, C, s);
  Band band;
  bool done = kFewTop * k <= 2 * C * kRowThreads && F.collect_top(k, own, band);
  if (!done) {
    if (kFewTop * k <= 2 * C * kRowThreads) F.clear();
    F.sl.each([&](float z, int) {
      if (z >= kNegMax) atomicAdd(&F.hist(F.sub)[max(F.sc.template bin<true>(z), 0)], 1u);
    });
    __syncthreads();
    F.template merge<false>(kBins);
    if (!F.template find_bins<false>(static_cast<float>(k), band)) {
      F.set_band(band, 0, kBins - 1);
    } else if (S.before + static_cast<int>(S.total[band.hi]) > kCap) {
      __syncthreads();
      F.cut(band, kByCount, k, false, kNegMax, nullptr);
      F.clear();
      F.set_band(band, 0, kBins - 1);
      band.elo = F.zc;
    }
    __syncthreads();
    band.lo = 0;
    band.ehi = pos_inf();
    F.collect(band);
  }
  const int n = F.collected();
  if (rank == 0) F.pull(n);
  F.sync_all();  // the other CTAs' lists have been read
  if (rank != 0) return;
  const uint64_t* list = F.list();
  F.sort(F.list(), n);
  for (int j = threadIdx.x; j < k; j += kRowThreads) {
    P.ids[row * k + j] = j < n ? token_index(list[j]) : -1;
    P.values[row * k + j] = j < n ? token_logit(list[j]) : neg_inf();
  }
  if (threadIdx.x == 0) {
    double t = 0;
    for (int r = 0; r < C; ++r) t += S.xexp[r];
    if (P.lse) P.lse[row] = static_cast<float>(static_cast<double>(m) * P.invT + log(t));
    if (P.status) P.status[row] = 0;
  }
}

}  // namespace specv
