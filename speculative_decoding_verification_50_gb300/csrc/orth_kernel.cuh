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
  int32_t rows, cols, batch, blocks;  // blocks per matrix
  int32_t vec;                        // rows start at 16-byte boundaries
  const void* in;
  int64_t batch_stride, row_stride;
  ScaledSquares* part;                // [batch][blocks]
  // orth_scale_kernel
  uint16_t *hi, *lo;                  // [batch][rows][ld]
  int64_t ld;
  float scale;                        // X is kept times this
  float* norm;                        // optional [batch]
  int32_t* status;                    // optional [batch]
};

__device__ __forceinline__ float2 unpack_f16(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// Lanes hold rows: pairs of lanes swap, so that each stores two rows of one column.
__device__ __forceinline__ void put_mirror(uint16_t* to, int64_t ld, int n, int row, int lane, int col, const uint32_t (&w)[32]) {
  const int odd = lane & 1;
  uint16_t* out = to + (row & ~1);
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, w[j], 1);
    const uint32_t pair = odd ? (other >> 16) | (w[j] & 0xffff0000u) : (w[j] & 0xffffu) | (other << 16);
    const int r = col + 2 * j + odd;
    if (r < n && (row & ~1) < n) *reinterpret_cast<uint32_t*>(out + r * ld) = pair;
  }
}

// A symmetric matrix in fp16 from its upper tiles, alpha A B^T (ADD: + beta C), and (FINE)
// what fp16 leaves out.
template <bool ADD, bool FINE>
struct SymEpi : PlainEpi {
  static constexpr int kStaging = FINE ? 8192 : 4096;
  struct Params {
    Out16 hi, lo;
    uint16_t *mirror_hi, *mirror_lo;   // the matrices themselves
    CUtensorMap chi, clo;              // ADD: C (boxes of 64 x 32)
    int64_t ld, zstride;
    int32_t n;
    float alpha, beta;
  };
  static __device__ __forceinline__ void ahead(const Params& e, EpiTile& q) {
    if (ADD && q.row0 < e.n && q.col0 < e.n) fetch16<FINE>(&e.chi, &e.clo, q, q.col0);
  }
  static __device__ __forceinline__ void tile(const Params& e, EpiTile& q, State&) {
    if (q.row0 >= e.n) return;
    const int row = q.row0 + q.lane;
#pragma unroll 1
    for (int c = 0; c < kProdHalf; c += 64) {
      const int col = q.col0 + c;
      if (col >= e.n) break;
      uint32_t w[32], l[32];
      if (ADD) {
        if (c > 0) fetch16<FINE>(&e.chi, &e.clo, q, col);
        if (!fetched(q)) return;
        unstage16(q.staging, q.lane, w);
        if (FINE) unstage16(q.staging + 4096, q.lane, l);
        __syncwarp();
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[32];
        tmem_load32(q.tmem + c + 32 * h, v);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int k = 16 * h + j;
          float x = v[2 * j] * e.alpha, y = v[2 * j + 1] * e.alpha;
          if (ADD) {
            float2 f = unpack_f16(w[k]);
            if (FINE) {
              const float2 g = unpack_f16(l[k]);
              f.x += g.x, f.y += g.y;
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
      }
      if (FINE) {
        if (!ADD) {
          if (q.lane == 0) tma_wait_read<0>();
          __syncwarp();
        }
        put16_pair(e.hi, e.lo, q.staging, q.lane, q.row0, col, q.z, w, l);
      } else {
        put16(e.hi, q.staging, q.lane, q.row0, col, q.z, q.rows, w);
      }
      if (q.unit.m != q.unit.n) {
        put_mirror(e.mirror_hi + q.z * e.zstride, e.ld, e.n, row, q.lane, col, w);
        if (FINE) put_mirror(e.mirror_lo + q.z * e.zstride, e.ld, e.n, row, q.lane, col, l);
      }
    }
  }
};

// X' = a X + A B^T, as fp16 and what that leaves out, or (LAST) in bf16.
template <bool LAST>
struct StepEpi : PlainEpi {
  static constexpr int kStaging = 8192;
  struct Params {
    Out16 hi, lo;             // LAST: hi alone
    CUtensorMap xhi, xlo;     // X (boxes of 64 x 32)
    int32_t rows, cols;
    float alpha, beta;        // of the product, of X
  };
  static __device__ __forceinline__ void ahead(const Params& e, EpiTile& q) {
    if (q.row0 < e.rows && q.col0 < e.cols) fetch16<true>(&e.xhi, &e.xlo, q, q.col0);
  }
  static __device__ __forceinline__ void tile(const Params& e, EpiTile& q, State&) {
    if (q.row0 >= e.rows) return;
#pragma unroll 1
    for (int c = 0; c < kProdHalf; c += 64) {
      const int col = q.col0 + c;
      if (col >= e.cols) break;
      uint32_t w[32], l[32];
      if (c > 0) fetch16<true>(&e.xhi, &e.xlo, q, col);
      if (!fetched(q)) return;
      unstage16(q.staging, q.lane, w);
      unstage16(q.staging + 4096, q.lane, l);
      __syncwarp();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[32];
        tmem_load32(q.tmem + c + 32 * h, v);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float2 a = unpack_f16(w[16 * h + j]), b = unpack_f16(l[16 * h + j]);
          const float x = fmaf(a.x + b.x, e.beta, v[2 * j] * e.alpha), y = fmaf(a.y + b.y, e.beta, v[2 * j + 1] * e.alpha);
          if (LAST) {
            w[16 * h + j] = pack_bf16(x, y);
          } else {
            w[16 * h + j] = pack_f16(x, y);
            const float2 f = unpack_f16(w[16 * h + j]);
            l[16 * h + j] = pack_f16(x - f.x, y - f.y);
          }
        }
      }
      if (LAST)
        put16(e.hi, q.staging, q.lane, q.row0, col, q.z, q.rows, w);
      else
        put16_pair(e.hi, e.lo, q.staging, q.lane, q.row0, col, q.z, w, l);
    }
  }
};

}  // namespace specv
