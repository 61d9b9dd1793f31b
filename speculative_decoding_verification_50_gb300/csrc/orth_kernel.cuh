// An update's singular values drawn towards one by odd polynomials (Newton-Schulz):
//
//   X = G / |G|_F,  then per step  S = X X^T (X^T X where rows are the longer side),
//   P = b S + c S S,  X <- a X + P X (X P).
//
// What is rounded, and why it may be.  S, P and the X that the products read are fp16
// (2^-11 of an entry at most): a step treats a small singular direction by a X almost
// alone, and that term keeps X to 21 bits (fp16 and the fp16 of what that leaves out).
// With X in fp16 alone its rounding, spread over all directions, grows with the small
// ones, by a factor a per step: a low-rank update then ends 2e-2 off its exact result, in
// this form 2e-4 (random ones 1.5e-3; bf16 throughout 0.16 and 1e-2).  Sums are fp32.
// Those are matrices whose entries' roundings are independent.  Where they agree, S and P are
// off the same way in every direction: five rows that are not zero 3e-3 (one 4e-3), diagonal,
// constant and +-1 matrices up to 9e-3.
// Matrices whose smaller side is at most 256 (one tile) cost launches, not products, and
// errors of few singular values do not average out: there S and P are kept to 21 bits too,
// and products take three parts (high x high, high x low, low x high).
// Each matrix is kept times a power of two that leaves fp16 its range (from bounds on the
// singular values, on the host).
//
// S and P are symmetric: tiles on and above the diagonal are computed, and written twice.
#pragma once

#include "product_kernel.cuh"

namespace specv {

constexpr int kOrthThreads = 256;

// A sum of squares as s m^2, m a power of two no smaller than half of the largest entry.
struct ScaledSquares {
  float m, s;
};

struct OrthInParams {
  int64_t rows, cols;                 // (a matrix without gaps, also in X: one row)
  int32_t batch, blocks;              // blocks per matrix
  int32_t vec;                        // rows start at 16-byte boundaries
  const void* in;
  int64_t batch_stride, row_stride;
  ScaledSquares* part;                // [batch][blocks]
  // orth_scale_kernel
  uint16_t *hi, *lo;                  // [batch][rows][ld]
  int64_t ld, matrix;                 // strides of a row and a matrix
  float scale;                        // X is kept times this
  float* norm;                        // optional [batch]
  int32_t* status;                    // optional [batch]
};

__device__ __forceinline__ float2 unpack_f16(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// An epilogue warp's tile goes by groups of 32 columns through two buffers in shared
// memory: what a group reads (C, in fp16 and what that leaves out) comes into a buffer by
// TMA, its results replace it and leave by TMA, while the other buffer's group is under way.
// A lane's own loads and stores would touch a line per lane.  Boxes are 32 rows of 64
// bytes, in which 16-byte words are swapped by bits 1 and 2 of the row (TMA's 64-byte
// swizzle).
constexpr int kBox = 2048;

__device__ __forceinline__ uint32_t box_at(int lane, int j) { return lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4); }
__device__ __forceinline__ void box_put(uint8_t* box, int lane, const uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(box + box_at(lane, j)) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}
__device__ __forceinline__ void box_get(const uint8_t* box, int lane, uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 v = *reinterpret_cast<const uint4*>(box + box_at(lane, j));
    w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
  }
}
// The transposed box: lanes hold rows, so pairs of lanes swap, and each stores two rows of
// one column.  32 rows (columns of the box) of 64 bytes, not swizzled.
__device__ __forceinline__ void box_put_transposed(uint8_t* box, int lane, const uint32_t (&w)[16]) {
  const int odd = lane & 1;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, w[j], 1);
    const uint32_t pair = odd ? (other >> 16) | (w[j] & 0xffff0000u) : (w[j] & 0xffffu) | (other << 16);
    *reinterpret_cast<uint32_t*>(box + (2 * j + odd) * 64 + (lane >> 1) * 4) = pair;
  }
}

// The two buffers: group g uses buffer g & 1, of BUF bytes, and its barrier.
template <int BUF>
struct Boxes {
  // Both inputs of a group (lo: where LOW), by lane 0; the stores of the group before last,
  // which used the buffer, have read it.
  template <bool LOW>
  static __device__ __forceinline__ void fetch(const CUtensorMap* hi, const CUtensorMap* lo, EpiTile& q, int g, int col) {
    q.asked ^= 1u << (g & 1);
    if (q.lane == 0) {
      uint8_t* at = q.staging + (g & 1) * BUF;
      uint64_t* bar = q.bar + (g & 1);
      mbar_arrive_expect_tx(bar, (LOW ? 2 * kBox : kBox) + q.extra);
      tma_load<false>(smem_u32(at), hi, col, q.row0, q.z, smem_u32(bar));
      if (LOW) tma_load<false>(smem_u32(at) + kBox, lo, col, q.row0, q.z, smem_u32(bar));
    }
    q.extra = 0;
  }
  // The warp's wait for a group (false: it ran out).
  static __device__ __forceinline__ bool wait(EpiTile& q, int g) {
    const bool ok = __all_sync(0xffffffffu, prod_wait(q.bar + (g & 1), (q.phase >> (g & 1)) & 1, q.gone));
    if (ok) q.phase ^= 1u << (g & 1);
    return ok;
  }
};

// A symmetric matrix in fp16 from its tiles on and above the diagonal, alpha A B^T
// (ADD: + beta C), and (FINE) what fp16 leaves out.
template <bool ADD, bool FINE>
struct SymEpi : PlainEpi {
  static constexpr int kBuf = FINE ? 4 * kBox : 2 * kBox, kStaging = 2 * kBuf;  // hi, (lo,) and the transposed ones
  static constexpr bool kReads = ADD;
  using B = Boxes<kBuf>;
  struct Params {
    CUtensorMap hi, lo;                // boxes of 32 x 32, swizzled
    CUtensorMap mirror_hi, mirror_lo;  // the same matrices, boxes of 32 x 32, not swizzled
    CUtensorMap chi, clo;              // ADD: C
    int32_t n;
    float alpha, beta;
  };
  static __device__ __forceinline__ void ahead(const Params& e, EpiTile& q) {
    if (!ADD || q.row0 >= e.n) return;
    if (q.lane == 0) tma_wait_read<0>();
    if (q.col0 < e.n) B::template fetch<FINE>(&e.chi, &e.clo, q, 0, q.col0);
    if (q.col0 + 32 < e.n) B::template fetch<FINE>(&e.chi, &e.clo, q, 1, q.col0 + 32);
  }
  template <int COLS>
  static __device__ __forceinline__ void tile(const Params& e, EpiTile& q, State&) {
    if (q.row0 >= e.n) return;
#pragma unroll 1
    for (int g = 0; g < COLS / 32; ++g) {
      const int col = q.col0 + 32 * g;
      if (col >= e.n) break;
      uint8_t* buf = q.staging + (g & 1) * kBuf;
      uint32_t w[16], l[16];
      if (ADD) {
        if (!B::wait(q, g)) return;
        box_get(buf, q.lane, w);
        if (FINE) box_get(buf + kBox, q.lane, l);
      } else {
        if (q.lane == 0) {  // (a tile before this one may have ended in either buffer)
          if (g == 0)
            tma_wait_read<0>();
          else
            tma_wait_read<1>();
        }
      }
      __syncwarp();
      float v[32];
      tmem_load32(q.tmem + 32 * g, v);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        float x = v[2 * k] * e.alpha, y = v[2 * k + 1] * e.alpha;
        if (ADD) {
          float2 f = unpack_f16(w[k]);
          if (FINE) {
            const float2 d = unpack_f16(l[k]);
            f.x += d.x, f.y += d.y;
          }
          x = fmaf(f.x, e.beta, x);
          y = fmaf(f.y, e.beta, y);
        }
        w[k] = pack_f16(x, y);
        if (FINE) {
          const float2 f = unpack_f16(w[k]);
          l[k] = pack_f16(x - f.x, y - f.y);
        }
      }
      const bool mirror = q.unit.m != q.unit.n;
      box_put(buf, q.lane, w);
      if (FINE) box_put(buf + kBox, q.lane, l);
      if (mirror) {
        box_put_transposed(buf + kBuf / 2, q.lane, w);
        if (FINE) box_put_transposed(buf + kBuf / 2 + kBox, q.lane, l);
      }
      fence_async_shared();
      __syncwarp();
      if (q.lane == 0) {
        tma_store(&e.hi, col, q.row0, q.z, smem_u32(buf));
        if (FINE) tma_store(&e.lo, col, q.row0, q.z, smem_u32(buf) + kBox);
        if (mirror) {
          tma_store(&e.mirror_hi, q.row0, col, q.z, smem_u32(buf) + kBuf / 2);
          if (FINE) tma_store(&e.mirror_lo, q.row0, col, q.z, smem_u32(buf) + kBuf / 2 + kBox);
        }
        tma_commit();
      }
      // (the group before this one has left its buffer: the next one's input)
      if (ADD && g >= 1 && g + 1 < COLS / 32 && col + 32 < e.n) {
        if (q.lane == 0) tma_wait_read<1>();
        B::template fetch<FINE>(&e.chi, &e.clo, q, g + 1, col + 32);
      }
    }
  }
};

// S from parts of K that were summed apart (tiles on and above the diagonal): a patch of
// 64 x 64 per CTA, and its transposed.  Bound by bytes.
struct OrthJoinParams {
  int32_t n, splits, patches;   // patches along a side
  const float* sum;             // [batch][splits][n][ld]
  uint16_t *hi, *lo;            // [batch][n][ld]; lo: optional
  int64_t ld;
  float alpha;
};

// X' = a X + A B^T, as fp16 and what that leaves out, or (LAST) in bf16.
template <bool LAST>
struct StepEpi : PlainEpi {
  static constexpr int kBuf = 2 * kBox, kStaging = 2 * kBuf;
  static constexpr bool kReads = true;
  using B = Boxes<kBuf>;
  struct Params {
    CUtensorMap hi, lo;       // LAST: hi alone
    CUtensorMap xhi, xlo;     // X
    uint16_t* direct;         // LAST, not null: out's rows do not start at 16-byte boundaries
    int64_t stride, zstride;  // of direct
    int32_t rows, cols;
    float alpha, beta;        // of the product, of X
  };
  static __device__ __forceinline__ void ahead(const Params& e, EpiTile& q) {
    if (q.row0 >= e.rows) return;
    if (q.lane == 0) tma_wait_read<0>();
    if (q.col0 < e.cols) B::template fetch<true>(&e.xhi, &e.xlo, q, 0, q.col0);
    if (q.col0 + 32 < e.cols) B::template fetch<true>(&e.xhi, &e.xlo, q, 1, q.col0 + 32);
  }
  template <int COLS>
  static __device__ __forceinline__ void tile(const Params& e, EpiTile& q, State&) {
    if (q.row0 >= e.rows) return;
#pragma unroll 1
    for (int g = 0; g < COLS / 32; ++g) {
      const int col = q.col0 + 32 * g;
      if (col >= e.cols) break;
      uint8_t* buf = q.staging + (g & 1) * kBuf;
      uint32_t w[16], l[16];
      if (!B::wait(q, g)) return;
      box_get(buf, q.lane, w);
      box_get(buf + kBox, q.lane, l);
      __syncwarp();
      float v[32];
      tmem_load32(q.tmem + 32 * g, v);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float2 a = unpack_f16(w[k]), b = unpack_f16(l[k]);
        const float x = fmaf(a.x + b.x, e.beta, v[2 * k] * e.alpha), y = fmaf(a.y + b.y, e.beta, v[2 * k + 1] * e.alpha);
        if (LAST) {
          w[k] = pack_bf16(x, y);
        } else {
          w[k] = pack_f16(x, y);
          const float2 f = unpack_f16(w[k]);
          l[k] = pack_f16(x - f.x, y - f.y);
        }
      }
      box_put(buf, q.lane, w);
      if (!LAST) box_put(buf + kBox, q.lane, l);
      fence_async_shared();
      __syncwarp();
      if (!LAST || !e.direct) {
        if (q.lane == 0) {
          tma_store(&e.hi, col, q.row0, q.z, smem_u32(buf));
          if (!LAST) tma_store(&e.lo, col, q.row0, q.z, smem_u32(buf) + kBox);
          tma_commit();
        }
      } else {  // half a warp per row
        const int n = min(e.rows - q.row0, 32), width = min(e.cols - col, 32), c = 2 * (q.lane & 15);
        uint16_t* out = e.direct + q.z * e.zstride + static_cast<int64_t>(q.row0) * e.stride + col;
        for (int r = q.lane >> 4; r < n; r += 2) {
          const uint32_t x = *reinterpret_cast<const uint32_t*>(buf + box_at(r, (q.lane & 15) >> 2) + (q.lane & 3) * 4);
          if (c < width) out[r * e.stride + c] = static_cast<uint16_t>(x);
          if (c + 1 < width) out[r * e.stride + c + 1] = static_cast<uint16_t>(x >> 16);
        }
        __syncwarp();
      }
      if (g >= 1 && g + 1 < COLS / 32 && col + 32 < e.cols) {
        if (q.lane == 0) tma_wait_read<1>();
        B::template fetch<true>(&e.xhi, &e.xlo, q, g + 1, col + 32);
      }
    }
  }
};

}  // namespace specv
