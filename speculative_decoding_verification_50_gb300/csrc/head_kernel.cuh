// The cross entropy of given tokens from hidden states h [N, D] and the head W [V, D],
// and its gradients, without the logits as an input or an output.
//
//   z = s h W^T,  nll_i = log(1 + sum_{v != t} exp(z_iv - z_it)),  lse_i = z_it + nll_i,
//   dz_iv = g_i exp(z_iv - lse_i), at the target g_i (exp(-nll_i) - 1),
//   dh = s dz W,  dW = s dz^T h.
//
// The target's logit is left out of the sums, so that the loss and the gradient at the
// target keep their digits where the row is nearly certain.  The forward pass keeps, per
// row and 128 (few rows: 64) columns, the largest logit and the sum relative to it; a second
// kernel joins them.  The backward pass computes the logits again, a piece of the
// vocabulary at a time, turns them into dz (bf16, as the products that read it want it:
// each element is off by at most 2^-8 of itself) and multiplies that by W and by h.
// Rows that count for nothing (no target, weight 0) are left out of every product: the
// others are gathered first.
#pragma once

#include "product_kernel.cuh"

namespace specv {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Logits far from zero.  An exponent z s log2(e) - m s log2(e) from two rounded products is off
// by 2^-24 of their size, not of its own: where the largest logit is above kFar (in powers of
// two; 4e-6 of a sum there) the difference is taken first.  The probabilities of a row whose
// log-sum-exp is above kFarRow (1e-4 of them there) are taken relative to a logit of the row.
// Warps with such a row take a loop that chooses by row: a row's bits do not depend on its
// neighbours.
constexpr float kFar = 128.f, kFarRow = 2048.f;

// What the backward pass knows of a row: its probabilities are 2^((z - ref) s log2(e) - off).
struct alignas(16) HeadRow {
  float ref;   // 0, or, in rows far from zero, the largest logit or the target's (an accumulator)
  float off;   // (lse - s ref) log2(e)
  float g;     // upstream weight x s, over the call's largest (HeadRowsParams::most); 0: no gradient
  float at;    // dz at the target
  int32_t target;
  float most;  // of its exponents: 0 in rows far from zero, whatever their statistics hold, else infinity
  int32_t none[2];
};
__device__ __forceinline__ HeadRow head_no_row() { return {0.f, 0.f, 0.f, 0.f, -1, pos_inf(), {0, 0}}; }

// (smallest of three, NaN ignored)
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

struct HeadStatsParams {
  const int32_t* target;  // [rows], -1: none
  float2* part;           // [ceil(V / PART)][ld]: largest accumulator, sum relative to it
  float* z_target;        // [rows]: the target's accumulator
  int64_t ld;
  int32_t V;
  float c2;               // s log2(e)
};

// The forward pass over a tile: 3.5 operations an element (maximum, minimum and NaN of
// pairs, one fused multiply-add, one exponential, one addition), under the products of
// the next tile.  The tensor core cuts each sum off (towards zero), so that the error of a
// long sum grows with its length: sums over more than kStatsChunk blocks of K are taken in
// chunks, which are added here (LONG; D = 4096: 2.3e-6 of the loss in one sum, 5e-7 in
// chunks of 16 blocks).  Rows of one tile, bound by the head's bytes, take shorter ones
// (45 x 4096 x 128256: 176 us in chunks of 8 blocks, 179 of 4, 194 of 2; 2e-7, 1e-7 and 1e-7
// off).  PART: columns per partial sum, those of an epilogue warp.  A lane's 128 sums (LONG, PART
// 128) do not all fit beside the rest in its registers: 40 bytes are spilled here and 60 in
// KeepEpi<128> (120 and 156 read back), the only product kernels with spills.
constexpr int kStatsChunk = 16, kStatsChunkFew = 4;
template <bool LONG, int PART>
struct StatsEpi : PlainEpi {
  static constexpr bool kChunks = LONG;
  struct State {
    float v[LONG ? PART : 1];
  };
  static __device__ __forceinline__ void start(State& sum) {
    if constexpr (LONG) {
#pragma unroll
      for (int j = 0; j < PART; ++j) sum.v[j] = 0.f;
    }
  }
  static __device__ __forceinline__ void add(EpiTile& q, State& sum) {
    if constexpr (LONG) {
#pragma unroll
      for (int c = 0; c < PART; c += 32) {
        float v[32];
        tmem_load32(q.tmem + c, v);
#pragma unroll
        for (int j = 0; j < 32; ++j) sum.v[c + j] += v[j];
      }
    }
  }
  static constexpr int kStaging = 0;
  using Params = HeadStatsParams;
  // 32 columns: `at` is the target's place among them, `left` of them are the vocabulary's;
  // mine: whether the lane has a row (what others hold may be anything).
  static __device__ __forceinline__ void part32(const Params& e, float (&v)[32], int i, bool mine, int at, int left, float& m,
                                                float (&s)[4], bool& bad) {
    if (left <= 0) return;
    float hi = v[0], lo = v[0];
#pragma unroll
    for (int j = 1; j < 31; j += 2) {
      hi = max3_nan(hi, v[j], v[j + 1]);
      lo = min3(lo, v[j], v[j + 1]);
    }
    hi = max3_nan(hi, v[31], v[31]);
    lo = fminf(lo, v[31]);
    bad |= !(hi < pos_inf()) || !(lo > neg_inf());
    if (__any_sync(0xffffffffu, static_cast<unsigned>(at) < 32u) || left < 32) {
      hi = neg_inf();
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        if (j == at) e.z_target[i] = v[j];
        if (j == at || j >= left) v[j] = neg_inf();
        hi = fmaxf(hi, v[j]);
      }
    }
    if (hi > m) {
      const float f = ex2((m - hi) * e.c2);
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] *= f;
      m = hi;
    }
    const float mc = -m * e.c2;
    const bool far = fabsf(mc) > kFar && hi > neg_inf() && mine;
    if (__any_sync(0xffffffffu, far)) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        s[j & 3] += far ? ex2((v[j] - m) * e.c2) : hi > neg_inf() ? ex2(fmaf(v[j], e.c2, mc)) : 0.f;
    } else if (hi > neg_inf()) {
#pragma unroll
      for (int j = 0; j < 32; ++j) s[j & 3] += ex2(fmaf(v[j], e.c2, mc));
    }
  }
  template <int COLS>
  static __device__ __forceinline__ void tile(const Params& e, EpiTile& q, State& sum) {
    if (q.row0 >= q.rows || q.col0 >= e.V) return;
    const int i = q.row0 + q.lane;
    const int target = i < q.rows ? e.target[i] : -1;
    float m = kNegMax, s[4] = {0.f, 0.f, 0.f, 0.f};
    bool bad = false;
#pragma unroll(LONG ? PART / 32 : 1)
    for (int c = 0; c < PART; c += 32) {
      float v[32];
      if constexpr (LONG) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = sum.v[c + j];
      } else {
        tmem_load32(q.tmem + c, v);
      }
      part32(e, v, i, i < q.rows, target - (q.col0 + c), e.V - (q.col0 + c), m, s, bad);
    }
    const float total = (s[0] + s[1]) + (s[2] + s[3]);
    if (i < q.rows) e.part[static_cast<int64_t>(q.col0 / PART) * e.ld + i] = make_float2(m, bad ? __int_as_float(0x7fc00000) : total);
  }
};

// The forward pass where the gradients follow in the same call and the weights exp(z - m),
// m a row's largest logit of PART columns, are kept for them: times 2^15 in fp16 (off by 2^-11
// of a weight at most, and by 2^-40 of the largest of PART), so that the logits need no second
// product (4096 x 4096 x 128256, 0.7 of the rows in use: 6.0 ms, 7.7 with it).
constexpr float kKeepScale = 15.f;         // (its logarithm)
constexpr float kUnkeep = 1.f / 32768.f;
template <int PART>
struct KeepEpi : StatsEpi<true, PART> {
  static constexpr int kStaging = 4096;
  struct Params {
    HeadStatsParams s;
    Out16 out;
  };
  template <int COLS>
  static __device__ __forceinline__ void tile(const Params& e, EpiTile& q, typename StatsEpi<true, PART>::State& sum) {
    if (q.row0 >= q.rows || q.col0 >= e.s.V) return;
    const int i = q.row0 + q.lane, at = (i < q.rows ? e.s.target[i] : -1) - q.col0, left = e.s.V - q.col0;
    float hi = sum.v[0], lo = sum.v[0];
#pragma unroll
    for (int j = 1; j < PART - 1; j += 2) {
      hi = max3_nan(hi, sum.v[j], sum.v[j + 1]);
      lo = min3(lo, sum.v[j], sum.v[j + 1]);
    }
    hi = max3_nan(hi, sum.v[PART - 1], sum.v[PART - 1]);
    lo = fminf(lo, sum.v[PART - 1]);
    const bool bad = !(hi < pos_inf()) || !(lo > neg_inf());
    if (__any_sync(0xffffffffu, static_cast<unsigned>(at) < static_cast<unsigned>(PART)) || left < PART) {
      hi = neg_inf();
#pragma unroll
      for (int j = 0; j < PART; ++j) {
        if (j == at) e.s.z_target[i] = sum.v[j];
        if (j == at || j >= left) sum.v[j] = neg_inf();
        hi = fmaxf(hi, sum.v[j]);
      }
    }
    const float m = fmaxf(hi, kNegMax), mc = kKeepScale - m * e.s.c2;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    const bool far = fabsf(m * e.s.c2) > kFar && i < q.rows;
    if (__any_sync(0xffffffffu, far)) {
#pragma unroll
      for (int j = 0; j < PART; ++j) sum.v[j] = ex2(fmaf(far ? sum.v[j] - m : sum.v[j], e.s.c2, far ? kKeepScale : mc));
    } else {
#pragma unroll
      for (int j = 0; j < PART; ++j) sum.v[j] = ex2(fmaf(sum.v[j], e.s.c2, mc));
    }
#pragma unroll
    for (int j = 0; j < PART; ++j) s[j & 3] += sum.v[j];
    const float total = hi > neg_inf() ? ((s[0] + s[1]) + (s[2] + s[3])) * kUnkeep : 0.f;
    if (i < q.rows)
      e.s.part[static_cast<int64_t>(q.col0 / PART) * e.s.ld + i] = make_float2(m, bad ? __int_as_float(0x7fc00000) : total);
#pragma unroll
    for (int c = 0; c < PART; c += 64) {
      uint32_t w[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) w[j] = pack_f16(sum.v[c + 2 * j], sum.v[c + 2 * j + 1]);
      put16(e.out, q.staging, q.lane, q.row0, q.col0 + c, 0, q.rows, w);
    }
  }
};

// dz of a tile in bf16.
struct ProbEpi : PlainEpi {
  static constexpr int kStaging = 4096;
  struct Params {
    Out16 out;
    const HeadRow* row;  // [rows]
    int32_t first;       // the piece's first token
    float c2;
  };
  template <int COLS>
  static __device__ __forceinline__ void tile(const Params& e, EpiTile& q, State&) {
    // (the rows up to a multiple of 64 are read along K by the product for dW: zeros)
    const int rows = max((q.rows + kProdBK - 1) / kProdBK * kProdBK, kProdBK);
    if (q.row0 >= rows) return;
    const int i = q.row0 + q.lane;
    HeadRow r = head_no_row();
    if (i < q.rows) {
      const float4 x = *reinterpret_cast<const float4*>(e.row + i);
      r.ref = x.x, r.off = x.y, r.g = x.z, r.at = x.w, r.target = e.row[i].target, r.most = e.row[i].most;
    }
    const bool far = __any_sync(0xffffffffu, r.most == 0.f);
#pragma unroll 1
    for (int c = 0; c < COLS; c += 64) {
      if (q.col0 + c >= e.out.cols) break;
      uint32_t w[32];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[32];
        tmem_load32(q.tmem + c + 32 * h, v);
        if (far) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = r.g * ex2(fminf(fmaf(v[j] - r.ref, e.c2, -r.off), r.most));
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = r.g * ex2(fmaf(v[j], e.c2, -r.off));
        }
        const int at = r.target - e.first - (q.col0 + c + 32 * h);
        if (__any_sync(0xffffffffu, static_cast<unsigned>(at) < 32u || r.g == 0.f)) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = r.g == 0.f ? 0.f : j == at ? r.at : v[j];
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) w[16 * h + j] = pack_bf16(v[2 * j], v[2 * j + 1]);
      }
      put16(e.out, q.staging, q.lane, q.row0, q.col0 + c, 0, rows, w);
    }
  }
};

// Joins a maximum and a sum relative to it (sums of nothing: kNegMax, 0).
__device__ __forceinline__ void soft_join(float& m, float& s, float m2, float s2, float c) {
  const float M = fmaxf(m, m2);
  s = s * ex2((m - M) * c) + s2 * ex2((m2 - M) * c);
  m = M;
}

// ---- rows

struct HeadRowsParams {
  int32_t N, V;
  int32_t all;             // rows without a target count too
  const int32_t* target;
  const float* weight;     // optional
  const float* up;         // optional (backward)
  const float* stats;      // backward: [N, 2]; forward: null
  float scale;
  // The largest |g| of the rows (1 where none counts, or it is not finite).  dz is kept over
  // it, and the products of dz are multiplied by it in fp32: rows of one weight then have
  // -(1 - p) at their targets, which bf16 holds where p is small, in the place of a weight
  // like 1 / 2870 whose rounding every row would share (2e-3 of the gradients).
  float* most;
  int32_t* count;          // rows in use
  int32_t* place;          // [N]: a row's place among those in use, or -1
  int32_t* source;         // [N]: and back
  int32_t* use_target;     // [N], by place
  HeadRow* row;            // [N], by place (backward)
};

constexpr int kRowsThreads = 1024;

struct HeadGatherParams {
  HeadRowsParams info;     // info.row not null: rows are where they are, and what is known of them is written
  int32_t N, D, pad_to;    // rows up to a multiple of pad_to behind those in use are zeros
  int32_t vec;             // source rows start at 16-byte boundaries
  int32_t* bad;            // optional [N], by place: 1 for a row with an entry that is not finite; it becomes zeros
  const int32_t* count;    // optional: rows in use
  const int32_t* source;   // optional: by place
  const uint16_t* in;
  int64_t in_stride;
  uint16_t* out;
  int64_t out_stride;      // a multiple of 8
  // backward: the target's logit of rows far from zero, which what is known of them refers to
  const float* stats;      // [N, 2]; null: none
  const int32_t* target;   // by place
  HeadRow* row;            // by place
  const uint16_t* head;    // rows that need not be aligned
  int64_t head_stride;
  int32_t* late;           // optional: the call's word for late products, which begins as 0
};

constexpr int kGatherThreads = 256;

struct HeadJoinParams {
  int32_t N, V, parts;
  const float2* part;
  const float* z_target;
  int64_t ld;
  float scale;
  const int32_t* place;    // optional (null: a row is where it is)
  int32_t all;             // HeadRowsParams
  const int32_t* target;
  const float* weight;     // optional
  const int32_t* bad;      // optional, by place: rows with entries that are not finite
  const float* most;       // HeadRowsParams (where row is given)
  const int32_t* err;      // [errs] of the forward pass
  int32_t errs;
  float* loss;
  float* stats;            // [N, 2]
  int32_t* status;         // optional
  HeadRow* row;            // optional, by place: what the gradient's kernels read
};

constexpr int kJoinThreads = 256;

struct HeadWeightParams {
  int32_t N, V;
  const int32_t* count;    // optional: rows in use
  const float2* part;
  int64_t ld;
  const HeadRow* row;
  float c2;
  int32_t part_cols;       // columns per part
  uint16_t* w;             // [rows up to a block][stride]: weights in, dz out
  int64_t stride;
};

// The end of a call's gradients: dh (if any) from its sums; and where a product's wait ran out,
// zeros in the place of all of them, and the status.
struct HeadFinishParams {
  int32_t N, V, D, splits;
  const int32_t* late;
  int32_t* status;         // optional [N]: added to
  uint16_t* head;          // dW, optional
  int64_t head_stride;
  const float* sum;        // [splits][rows][ld]
  int64_t ld, split_stride;
  const int32_t* place;    // optional
  const HeadRow* row;      // by place
  const float* most;       // HeadRowsParams
  uint16_t* out;           // dh, optional
  int64_t stride;
  int32_t vec;
};

}  // namespace specv
