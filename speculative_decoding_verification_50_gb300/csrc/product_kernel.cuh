// Matrix products on the tensor cores with a fused epilogue: C = A B^T over tiles of
// 256 x 256, for the head's loss and for orthogonalised updates.
//
// A pair of CTAs (one cluster, two SMs) computes a tile with tcgen05.mma.cta_group::2:
// each CTA brings 128 rows of A and 128 rows of B, so that each operand byte that is loaded
// serves both SMs, and holds 128 rows of the fp32 accumulator in its tensor memory.  The
// accumulator has two stages of 256 columns: the epilogue of one tile runs under the
// products of the next.  Warps of a CTA: 0 loads, 1 issues the products (in the first CTA of
// the pair), 2 and 3 only fill their warpgroup, 4-11 epilogue (warp w reads tensor memory
// lanes 32 (w % 4), columns 128 (w / 4 - 1)).  The first warps are the oldest, which their
// scheduler prefers: the issue of products does not wait behind busy epilogue warps.  Groups
// of CTAs take tiles in a fixed order, so that results do not depend on timing.
//
// Operands are 16-bit, either "K-major" (rows of A or B contiguous along K) or
// "MN-major" (contiguous along M or N: the transposed matrix as it lies in memory), in
// shared memory under the 128-byte swizzle that TMA writes and the tensor core reads.
// A tile's K is cut into blocks of 64; TMA fills what lies outside of a matrix with zeros.
//
// What bounds it: a block of K is 512 cycles of the tensor core for 32 KB into each SM, 64
// bytes a clock, which is what an SM takes in from L2: blocks take 590 to 620 (tensor pipe
// 78 to 86 % active), 1.8 to 1.95 PFLOP/s for 4096 x 4096 x 32768 in one launch (of 1.92
// that a library's product measured); in long runs the clock falls to the power limit.
// A tile of its own per CTA (PAIR false) takes in the same bytes for half the work.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "specv_common.cuh"

namespace specv {

constexpr int kProdTile = 256;              // rows and columns of a cluster's tile
constexpr int kProdHalf = kProdTile / 2;    // rows of A, and of B, that one CTA loads
constexpr int kProdBK = 64;                 // K per stage: 128 bytes, the width of the swizzle
constexpr int kProdEpiWarps = 8;
constexpr int kProdThreads = 32 * (kProdEpiWarps + 4);
constexpr int kLoadWarp = 0, kMmaWarp = 1, kEpiWarp = 4;  // the first epilogue warp
// Registers a thread: launched with at most 168 (12 warps), of which the first four warps
// give up most to the epilogue's: 2 x 216 + 72 = 3 x 168.
constexpr int kEpiRegs = 216, kLoadRegs = 72;
constexpr int kOperandBytes = kProdHalf * kProdBK * 2;  // 16 KB
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kProdBarrierBytes = 512;
constexpr int kProdSmemMost = 227 * 1024;

// Stages that fit beside STAGING bytes per epilogue warp, and all of a CTA's bytes.
template <int STAGING>
constexpr int kProdStages = (kProdSmemMost - 1024 - kProdBarrierBytes - kProdEpiWarps * STAGING) / kStageBytes;
template <int STAGING>
constexpr int kProdSmem = 1024 + kProdBarrierBytes + kProdEpiWarps * STAGING + kProdStages<STAGING> * kStageBytes;

struct ProductParams {
  CUtensorMap a, b;
  CUtensorMap a_low, b_low;  // fine: what a and b leave out
  int32_t fine;              // C = A B^T + A B_low^T + A_low B^T, one after the other
  int32_t M, N, K;         // the largest sizes (host), N exact
  int32_t a_rows;          // not PAIR, A K-major: rows of A's boxes (0: all 128), where M has no more
  const int32_t* rows;     // device: the number of rows in use, in the place of M (rows_k: of K)
  int32_t rows_k;
  int32_t tn;              // tiles along N
  int32_t batch, splits;   // splits: parts of K that are summed apart
  int32_t chunk;           // blocks of K per accumulator (0: all): the epilogue adds up several
  int32_t symmetric;       // M == N, C symmetric: only tiles on and above the diagonal
  int32_t bf16;            // operands: bf16, or fp16
  uint32_t idesc;          // (set by the launch)
  int32_t* err;            // [clusters]: 0, or 1 where a wait ran out
  int32_t* status;         // optional [status_n]: a wait that ran out is added (kTimeout)
  int32_t status_n;
  int32_t* late;           // optional: one word, made 1 by a wait that ran out
  int32_t stall;           // test hook: 1 + the unit whose first copy is late
  int32_t stall_read;      // and 1 + that whose epilogue's first copy is
};

// Instruction descriptor of tcgen05.mma kind::f16 for tiles of tile x tile, fp32 accumulators.
constexpr uint32_t prod_idesc(bool bf16, bool a_mn, bool b_mn, int tile = kProdTile) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(tile >> 3) << 17) | (static_cast<uint32_t>(tile >> 4) << 24);
}

// ---- instructions

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The shared::cluster address of `addr` in the cluster's first CTA.
__device__ __forceinline__ uint32_t in_first_cta(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
// An arrival that hands over tensor memory alone (its loads are complete, and fenced): with
// the cluster's scope the release would wait for the warp's stores to global memory too,
// about 2600 cycles.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// A box into this CTA's shared memory; its bytes count on `bar`, which may be the pair's other CTA's.
template <bool PAIR>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  if (!PAIR) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
    return;
  }
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap* map, int x, int y, int z, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}
__device__ __forceinline__ void tma_add(const CUtensorMap* map, int x, int y, int z, uint32_t src) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}
__device__ __forceinline__ void tma_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void tma_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(LEFT) : "memory");
}
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void tmem_alloc_all(uint32_t at) {
  if (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(at) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(at) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}
template <bool PAIR>
__device__ __forceinline__ void tmem_free_all(uint32_t tmem) {
  if (PAIR)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
template <bool PAIR>
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  if (!PAIR) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
        : "memory");
    return;
  }
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
}
// Arrives on the barrier (PAIR: at this offset in both CTAs) once the products issued so far
// are done.
template <bool PAIR>
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  if (!PAIR) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
    return;
  }
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// The same, on this CTA's barrier alone.
template <bool PAIR>
__device__ __forceinline__ void tc_commit_own(uint32_t bar) {
  if (PAIR)
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
  else
    tc_commit<false>(bar);
}
// 32 columns of this warp's 32 lanes: thread l gets row l.
__device__ __forceinline__ void tmem_load32(uint32_t at, float (&v)[32]) {
  uint32_t* u = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(at)
      : "memory");
}

// Shared-memory descriptor of an operand under the 128-byte swizzle (version 1, layout
// type 2).  K-major: groups of 8 rows are 1024 bytes apart.  MN-major: a group of 64
// along M or N is [64 (K)][128 bytes]; groups of 8 along K are 1024 bytes apart, groups
// of 64 along M or N 8192.
template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  constexpr uint64_t lead = MN ? (kProdBK * 128) >> 4 : 1, stride = 1024 >> 4;
  return (static_cast<uint64_t>(addr >> 4) & 0x3fff) | (lead << 16) | (stride << 32) | (1ull << 46) | (2ull << 61);
}
// The step from 16 of K to the next, in the descriptor's 16-byte units.
template <bool MN>
constexpr uint64_t kOperandStep = MN ? (16 * 128) >> 4 : (16 * 2) >> 4;

// ---- units of work

struct Unit {
  int m, n, z, split, k0, k1;  // first row, first column, matrix, blocks of K
};

struct Units {
  int tile, tm, tn, per, span, blocks, count, splits, symmetric;  // span: blocks of K; blocks: with the parts of a fine product
  __device__ __forceinline__ Units(const ProductParams& p, int size) : tile(size) {
    int M = p.M, K = p.K;
    if (p.rows) (p.rows_k ? K : M) = *p.rows;
    // (without any row one tile is computed all the same: its zeros are read)
    tm = max((M + tile - 1) / tile, 1);
    tn = p.tn;
    splits = p.splits;
    symmetric = p.symmetric;
    span = max((K + kProdBK - 1) / kProdBK, 1);
    blocks = p.fine ? 3 * span : span;
    per = (symmetric ? tn * (tn + 1) / 2 : tm * tn) * splits;
    count = per * p.batch;
  }
  // A part of K after the other: clusters that run at the same time read the same slices of
  // A and B, which stay in L2 (4096 x 4096 x 32768 in three parts: 3.2 GB from HBM with
  // parts side by side, 1.4 so).  Rows in groups of 16 tiles, along which the tile index runs
  // first: clusters that run at the same time share columns of B, and the group's rows of A
  // stay in L2.
  __device__ __forceinline__ Unit at(int u) const {
    Unit r;
    r.z = u / per;
    int t = u - r.z * per;
    r.split = t / (per / splits);
    t -= r.split * (per / splits);
    int i, j;
    if (symmetric) {
      for (i = 0; t >= tn - i; ++i) t -= tn - i;
      j = i + t;
    } else {
      constexpr int kGroup = 16;
      const int g = t / (kGroup * tn), rows = min(tm - g * kGroup, kGroup);
      t -= g * kGroup * tn;
      i = g * kGroup + t % rows;
      j = t / rows;
    }
    r.m = i * tile;
    r.n = j * tile;
    r.k0 = static_cast<int>(static_cast<int64_t>(blocks) * r.split / splits);
    r.k1 = static_cast<int>(static_cast<int64_t>(blocks) * (r.split + 1) / splits);
    return r;
  }
};

// What an epilogue warp is given: its 32 rows (one per lane) and half of a tile's columns.
struct EpiTile {
  uint32_t tmem;      // of its first column
  uint8_t* staging;   // its own, 1024-byte aligned
  int row0, col0;     // its first row and column in C
  int z, split, lane;
  int rows;           // rows in use (M)
  Unit unit;
  uint64_t* bar;      // two of the warp's own, for what the epilogue reads, and their phases (bits)
  uint32_t phase;
  uint32_t asked;     // the phases that copies were asked for
  int extra;          // bytes that the next copy's wait is for beside the copy's (test hook)
  volatile int* gone;
};

// Whether a phase is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// A bounded wait (about two seconds); false once any wait of the CTA ran out.
__device__ __forceinline__ bool prod_wait(uint64_t* bar, uint32_t parity, volatile int* gone) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  for (uint32_t it = 0; it < (1u << 21); ++it) {
    if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
    if (*gone) return false;
    if (clock64() - t0 > 4000000000LL) break;
  }
  *gone = 1;
  return false;
}

// PAIR: a cluster of two CTAs per tile of 256 x 256; else a CTA per tile of 128 x 128, for
// products of few tiles (each operand byte then serves 128 rows, and L2 limits the rate).
template <bool PAIR, bool A_MN, bool B_MN, class Epi>
__global__ void __launch_bounds__(kProdThreads, 1)
    product_kernel(const __grid_constant__ ProductParams p, const __grid_constant__ typename Epi::Params e) {
  constexpr int S = kProdStages<Epi::kStaging>;  // 6 with a 4 KB box per epilogue warp
  extern __shared__ uint8_t raw[];
  uint8_t* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint8_t* staging = base + S * kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + kProdEpiWarps * Epi::kStaging);
  uint64_t *full = bars, *empty = bars + S, *tfull = bars + 2 * S, *tempty = tfull + 2, *drain = tempty + 2, *epi = drain + 1;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(epi + 2 * kProdEpiWarps);
  volatile int* gone = reinterpret_cast<volatile int*>(tmem_at + 1);
  static_assert((2 * S + 5 + 2 * kProdEpiWarps) * 8 + 8 <= kProdBarrierBytes, "barriers");

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  constexpr int kTile = PAIR ? kProdTile : kProdHalf, kCtas = PAIR ? 2 : 1;
  const uint32_t rank = PAIR ? cluster_rank() : 0;
  const int cluster = blockIdx.x / kCtas, clusters = gridDim.x / kCtas;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);   // the first CTA's loader; both CTAs' bytes
      mbar_init(&empty[s], 1);  // the products that read the stage
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tfull[s], 1);
      mbar_init(&tempty[s], kCtas * kProdEpiWarps);
    }
    mbar_init(drain, 1);
    for (int w = 0; w < 2 * kProdEpiWarps; ++w) mbar_init(&epi[w], 1);
    *gone = 0;
    fence_mbar_init();
    prefetch_map(&p.a);
    prefetch_map(&p.b);
  }
  if (warp == kMmaWarp) tmem_alloc_all<PAIR>(smem_u32(tmem_at));
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  pdl_wait_primary();
  pdl_launch_dependents();

  const Units units(p, kTile);
  if (warp == kLoadWarp) {  // ---- loads
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
    if (lane == 0) {
      // (rows of A that are not there take an SM's intake as others do, zeros or not: few rows
      // come in boxes of their own, and what lies in the rest of the buffer gives rows of C
      // that nothing reads)
      const int spare = !PAIR && !A_MN && p.a_rows ? (kProdHalf - p.a_rows) * kProdBK * 2 : 0;
      int it = 0;
      bool ok = true;
      for (int u = cluster; ok && u < units.count; u += clusters) {
        const Unit t = units.at(u);
        for (int k = t.k0; k < t.k1; ++k, ++it) {
          const int s = it % S;
          if (it >= S && !prod_wait(&empty[s], ((it / S) & 1) ^ 1, gone)) {
            ok = false;
            break;
          }
          if (rank == 0)
            mbar_arrive_expect_tx(&full[s], kCtas * kStageBytes - spare + ((p.stall == u + 1 && k == t.k0) ? 16 : 0));
          const uint32_t bar = PAIR ? in_first_cta(smem_u32(&full[s])) : smem_u32(&full[s]);
          const uint32_t sa = smem_u32(base + s * kStageBytes), sb = sa + kOperandBytes;
          const int part = p.fine ? k / units.span : 0;
          const CUtensorMap *pa = part == 2 ? &p.a_low : &p.a, *pb = part == 1 ? &p.b_low : &p.b;
          const int kk = (k - part * units.span) * kProdBK, m = t.m + static_cast<int>(rank) * kProdHalf, n = t.n + static_cast<int>(rank) * kProdHalf;
          if (A_MN) {
            tma_load<PAIR>(sa, pa, m, kk, t.z, bar);
            tma_load<PAIR>(sa + kOperandBytes / 2, pa, m + 64, kk, t.z, bar);
          } else {
            tma_load<PAIR>(sa, pa, kk, m, t.z, bar);
          }
          if (B_MN) {
            tma_load<PAIR>(sb, pb, n, kk, t.z, bar);
            tma_load<PAIR>(sb + kOperandBytes / 2, pb, n + 64, kk, t.z, bar);
          } else {
            tma_load<PAIR>(sb, pb, kk, n, t.z, bar);
          }
        }
      }
      // (a CTA leaves after every arrival at its barriers)
      for (int i = max(0, it - S); ok && i < it; ++i) ok = prod_wait(&empty[i % S], (i / S) & 1, gone);
      if (!ok && rank == 0) {  // copies in flight land before the CTAs leave
        const long long t0 = clock64();
        for (int i = max(0, it - S); i < it; ++i)
          while (!mbar_try_wait_sleep(&full[i % S], (i / S) & 1, 20000u) && clock64() - t0 < 1000000000LL) {
          }
      }
    }
  } else if (warp == kMmaWarp) {  // ---- products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
    if (lane == 0 && rank == 0) {
      // Whether the next block has landed is asked before the products of this one are
      // issued, and looked at after them: a wait between them leaves the tensor core idle.
      const uint64_t a0 = operand_desc<A_MN>(smem_u32(base)), b0 = operand_desc<B_MN>(smem_u32(base) + kOperandBytes);
      int n = 0, s = 0;
      uint32_t phase = 0;
      bool ok = true, landed = false, freed = true;
      const int chunk = Epi::kChunks && p.chunk ? p.chunk : 0x7fffffff;
      for (int u = cluster; ok && u < units.count; u += clusters) {
        const Unit t = units.at(u);
        for (int first = t.k0; ok && first < t.k1; first += min(chunk, t.k1 - first), ++n) {
          const int end = first + min(chunk, t.k1 - first);
          if (!freed && !prod_wait(&tempty[n & 1], ((n >> 1) & 1) ^ 1, gone)) {
            ok = false;
            break;
          }
          const uint32_t d = tmem + (n & 1) * kTile;
          for (int k = first; k < end; ++k) {
            if (!landed && !prod_wait(&full[s], phase, gone)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t da = a0 + s * (kStageBytes >> 4), db = b0 + s * (kStageBytes >> 4);
            uint64_t* emptied = &empty[s];
            if (++s == S) s = 0, phase ^= 1;
            landed = mbar_test(&full[s], phase);
            freed = n < 1 || mbar_test(&tempty[(n + 1) & 1], (((n + 1) >> 1) & 1) ^ 1);
#pragma unroll
            for (int j = 0; j < kProdBK / 16; ++j)
              tc_mma<PAIR>(d, da + j * kOperandStep<A_MN>, db + j * kOperandStep<B_MN>, p.idesc, k > first || j > 0);
            tc_commit<PAIR>(smem_u32(emptied));
          }
          if (ok) tc_commit<PAIR>(smem_u32(&tfull[n & 1]));
        }
      }
      // (products in flight end before tensor memory is freed, whatever other warps gave up on;
      // nothing waits for them at the pair's other CTA, which may leave)
      tc_commit_own<PAIR>(smem_u32(drain));
      const long long t0 = clock64();
      while (!mbar_try_wait_sleep(drain, 0, 20000u) && clock64() - t0 < 1000000000LL) {
      }
    }
  } else if (warp < kEpiWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
  } else {  // ---- epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    const int quarter = warp & 3, half = warp / 4 - 1;
    EpiTile q;
    q.staging = staging + (warp - kEpiWarp) * Epi::kStaging;
    q.lane = lane;
    q.rows = p.rows && !p.rows_k ? *p.rows : p.M;
    q.bar = &epi[2 * (warp - kEpiWarp)];
    q.phase = q.asked = 0;
    q.extra = 0;
    q.gone = gone;
    int n = 0;
    bool ok = true;
    typename Epi::State state;
    for (int u = cluster; ok && u < units.count; u += clusters) {
      const Unit t = units.at(u);
      q.row0 = t.m + static_cast<int>(rank) * kProdHalf + quarter * 32;
      q.col0 = t.n + half * (kTile / 2);
      q.z = t.z;
      q.split = t.split;
      q.unit = t;
      if (Epi::kReads && p.stall_read == u + 1) q.extra = 16;
      Epi::ahead(e, q);
      Epi::start(state);
      const int chunk = Epi::kChunks && p.chunk ? p.chunk : t.k1 - t.k0;
      for (int k = t.k0; k < t.k1; k += chunk, ++n) {
        const int acc = n & 1;
        q.tmem = tmem + acc * kTile + half * (kTile / 2) + (static_cast<uint32_t>(quarter * 32) << 16);
        ok = __all_sync(0xffffffffu, prod_wait(&tfull[acc], (n >> 1) & 1, gone));
        if (!ok) break;
        tc_fence_after();
        if (Epi::kChunks)
          Epi::add(q, state);
        else
          Epi::template tile<kTile / 2>(e, q, state);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(PAIR ? in_first_cta(smem_u32(&tempty[acc])) : smem_u32(&tempty[acc]));
        if (Epi::kReads && __any_sync(0xffffffffu, *gone)) {  // (what the next tile reads is not asked for)
          ok = false;
          break;
        }
      }
      if (Epi::kChunks && ok) Epi::template tile<kTile / 2>(e, q, state);
    }
    if (Epi::kReads && lane == 0) {  // copies asked for and not waited for land before the CTA leaves
      const long long t0 = clock64();
      for (int b = 0; b < 2; ++b)
        while ((((q.asked ^ q.phase) >> b) & 1) && !mbar_try_wait_sleep(q.bar + b, (q.phase >> b) & 1, 20000u) &&
               clock64() - t0 < 1000000000LL) {
        }
    }
    if (Epi::kStaging > 0 && lane == 0) tma_wait_read<0>();  // (the grid's end waits for the writes)
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_free_all<PAIR>(tmem);
  const int failed = *gone;
  if (threadIdx.x == 0 && p.err) p.err[blockIdx.x] = failed;
  if (failed && p.late && threadIdx.x == 0) *p.late = 1;
  if (failed && p.status)
    for (int i = threadIdx.x; i < p.status_n; i += kProdThreads) atomicOr(&p.status[i], kTimeout);
}

// ---- what epilogues share

// 64 columns of 16-bit values (pairs) of this lane's row into the warp's staging buffer,
// then out by TMA (`map`: boxes of 64 x 32 under the 128-byte swizzle), or, where C's rows
// do not start at 16-byte boundaries, row by row from shared memory.
struct Out16 {
  CUtensorMap map;
  uint16_t* direct;          // not null: stores without TMA
  int64_t stride, zstride;   // elements
  int32_t rows, cols;
};

__device__ __forceinline__ void stage16(uint8_t* staging, int lane, const uint32_t (&w)[32]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<uint4*>(staging + lane * 128 + ((j ^ (lane & 7)) << 4)) =
        make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}

// (rows: those of C in use; row0 and col0 of the 32 x 64 box; LEFT: stores that may still
// read other buffers)
template <int LEFT = 0>
__device__ __forceinline__ void put16(const Out16& o, uint8_t* staging, int lane, int row0, int col0, int z, int rows,
                                      const uint32_t (&w)[32]) {
  if (row0 >= rows || col0 >= o.cols) return;
  if (!o.direct) {
    if (lane == 0) tma_wait_read<LEFT>();
    __syncwarp();
    stage16(staging, lane, w);
    fence_async_shared();
    __syncwarp();
    if (lane == 0) {
      tma_store(&o.map, col0, row0, z, smem_u32(staging));
      tma_commit();
    }
    return;
  }
  __syncwarp();
  stage16(staging, lane, w);
  __syncwarp();
  const int n = min(rows - row0, 32);
  uint16_t* out = o.direct + z * o.zstride + static_cast<int64_t>(row0) * o.stride + col0;
  const int width = min(o.cols - col0, 64);
  for (int r = 0; r < n; ++r) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(staging + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
    if (2 * lane < width) out[r * o.stride + 2 * lane] = static_cast<uint16_t>(v);
    if (2 * lane + 1 < width) out[r * o.stride + 2 * lane + 1] = static_cast<uint16_t>(v >> 16);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// An epilogue of whole tiles that reads nothing of its own.
struct PlainEpi {
  struct State {};
  static constexpr bool kChunks = false, kReads = false;  // kReads: boxes (orth_kernel.cuh)
  template <typename P>
  static __device__ __forceinline__ void ahead(const P&, EpiTile&) {}
  static __device__ __forceinline__ void start(State&) {}
  static __device__ __forceinline__ void add(EpiTile&, State&) {}
};

// C = factor A B^T in bf16.  TWICE: two staging buffers, for products of so short a K that
// writing C bounds them (64 rows x 1024 x 32000: 23 us, with two 17).
template <bool TWICE>
struct StoreEpi : PlainEpi {
  static constexpr int kStaging = TWICE ? 8192 : 4096;
  struct Params {
    Out16 out;
    const float* factor;
  };
  template <int COLS>
  static __device__ __forceinline__ void tile(const Params& e, EpiTile& q, State&) {
    const float f = *e.factor;
#pragma unroll 1
    for (int c = 0; c < COLS; c += 64) {
      uint32_t w[32];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[32];
        tmem_load32(q.tmem + c + 32 * h, v);
#pragma unroll
        for (int j = 0; j < 16; ++j) w[16 * h + j] = pack_bf16(v[2 * j] * f, v[2 * j + 1] * f);
      }
      if (q.row0 >= q.rows || q.col0 + c >= e.out.cols) break;
      // (buffers in turn by the stores made: a tile may make one, two or none)
      put16<TWICE ? 1 : 0>(e.out, q.staging + (TWICE ? q.phase * 4096 : 0), q.lane, q.row0, q.col0 + c, q.z, q.rows, w);
      q.phase ^= 1;
    }
  }
};

// C in fp32 (boxes of 32 x 32), stored or added to what is there; a part of K (split)
// goes to its own matrix.
struct SumEpi : PlainEpi {
  static constexpr int kStaging = 4096;
  struct Params {
    CUtensorMap out;  // [batch x splits][rows][cols]
    int32_t cols;
    int32_t add;
    int32_t splits;
  };
  template <int COLS>
  static __device__ __forceinline__ void tile(const Params& e, EpiTile& q, State&) {
#pragma unroll 1
    for (int c = 0; c < COLS; c += 32) {
      float v[32];
      tmem_load32(q.tmem + c, v);
      if (q.row0 >= q.rows || q.col0 + c >= e.cols) continue;
      if (q.lane == 0) tma_wait_read<0>();
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<float4*>(q.staging + q.lane * 128 + ((j ^ (q.lane & 7)) << 4)) =
            make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      fence_async_shared();
      __syncwarp();
      if (q.lane == 0) {
        if (e.add)
          tma_add(&e.out, q.col0 + c, q.row0, q.z * e.splits + q.split, smem_u32(q.staging));
        else
          tma_store(&e.out, q.col0 + c, q.row0, q.z * e.splits + q.split, smem_u32(q.staging));
        tma_commit();
      }
    }
  }
};

}  // namespace specv
