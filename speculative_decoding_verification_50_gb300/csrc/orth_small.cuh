// All steps of an update whose smaller side is at most 128 in one kernel: the launches of
// the general path, a chain of three products a step, cost 8 us each whatever their size.
//
// A cluster of C CTAs holds a matrix Y [s, t] (the update, or its transposed) in shared
// memory, 128 columns per CTA, in fp16 and what that leaves out.  A step: each CTA's part of
// S = Y Y^T (tcgen05, one CTA each), summed over the cluster in a fixed order through
// distributed shared memory, 128 / C rows by each CTA, which hands its rows to all; then each
// CTA computes P = b S + c S S, and a Y + P Y of its own columns.  Products take three parts
// (high x high, high x low, low x high), as in the general path for such matrices.
// Bound by a chain: per step 2000 cycles for each of the three products, 5400 for the sum over
// the cluster (128 KB a CTA through distributed shared memory), 1900 for each of the two
// passes over tensor memory, 1700 for two cluster barriers.  128 x 512 bf16, five steps: 54 us
// (the general path 132).
#pragma once

#include "orth_kernel.cuh"

namespace specv {

constexpr int kSmallSide = 128;      // rows (s), and columns of a CTA
constexpr int kSmallThreads = 256;
constexpr int kSmallSteps = 32;
constexpr int kPlane = kSmallSide * kSmallSide * 2;  // one fp16 matrix: 32 KB
constexpr int kSmallSmem = 1024 + 6 * kPlane;        // Y, S (high and low), and sums in fp32 or P

struct SmallStep {
  float gram, poly, poly_s, step, step_y;  // factors of the products, and of S and Y beside them
};

struct SmallParams {
  int32_t s, t, steps;
  int32_t tall;                 // Y is the update's transposed
  int32_t vec;                  // rows of the update start at multiples of 4 elements' bytes
  int32_t out_vec;              // and those of out
  const void* in;
  int64_t batch_stride, row_stride;
  uint16_t* out;
  int64_t out_batch_stride, out_row_stride;
  float* norm;
  int32_t* status;
  float scale;                  // Y is kept times this at first
  int32_t stall;                // test hook: 1 + the matrix whose first products' end is not seen
  SmallStep step[kSmallSteps];
};

// Byte offset of element (row, col) of a 128 x 128 fp16 matrix: two panels of 64 columns,
// each K-major for its rows and MN-major for its columns under the 128-byte swizzle.
__device__ __forceinline__ uint32_t small_at(int row, int col) {
  return (col >> 6) * (kPlane / 2) + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4) + (col & 7) * 2;
}
// The same of a 128 x 128 matrix of fp32 sums (16-byte words of a row swapped by the row).
__device__ __forceinline__ uint32_t small_sum_at(int row, int word) { return row * 512 + ((word ^ (row & 31)) << 4); }

__device__ __forceinline__ uint32_t in_cta(uint32_t addr, int cta) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
  return r;
}
__device__ __forceinline__ float4 load_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void store_cluster(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

}  // namespace specv
