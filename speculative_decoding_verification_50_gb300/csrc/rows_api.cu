// C ABI of the operators that hold a row on chip (filtered sampling, top
// logits, distillation): argument checks, the row's split over a cluster, and
// the launch on the caller's stream.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "api.cuh"
#include "launch.cuh"

using namespace specv;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int elem_bytes(int32_t dtype) { return dtype == SPECV_BF16 ? 2 : 4; }

specv_status check_rows(const char* what, int32_t n, int32_t V, int32_t dtype) {
  if (n < 0) return api_fail(SPECV_ERR_INVALID_ARG, "%s=%d < 0", what, n);
  if (V < 1) return api_fail(SPECV_ERR_INVALID_ARG, "V=%d < 1", V);
  if (dtype != SPECV_BF16 && dtype != SPECV_FP32)
    return api_fail(SPECV_ERR_INVALID_ARG, "dtype=%d is not SPECV_BF16 or SPECV_FP32", dtype);
  return SPECV_OK;
}

constexpr size_t kSmemSm = 228 * 1024, kSmemCta = 227 * 1024, kSmemReserved = 1024;
constexpr size_t kDistillStatic = 2304;  // (at least what distill_kernel declares)

// The row's split over a cluster of C CTAs (a power of two) whose slices stay
// in shared memory beside `extra` bytes per CTA.  C is the smallest for which
// two CTAs fit an SM (one row's copies then run under the other's passes),
// and more while rows are too few to fill the SMs (us, against that smallest C:
// sampling 32 x 128256 bf16 under mixed rules 39.5, 41.4; 37 x 50257 35, 41).
// False: V does not fit.
bool split_row(int64_t rows, int32_t V, int32_t dtype, size_t extra, RowSplit& sp, size_t& smem) {
  const int vw = 16 / elem_bytes(dtype);
  const int64_t nvec = (static_cast<int64_t>(V) + vw - 1) / vw;
  const int64_t two = static_cast<int64_t>(kSmemSm / 2 - kSmemReserved - extra);
  const int64_t one = static_cast<int64_t>(kSmemCta - extra);
  auto segment = [&](int C) { return ((nvec + C - 1) / C + kRowWarps - 1) / kRowWarps; };
  auto slice = [&](int C) { return segment(C) * kRowWarps * 16; };
  int C = 1;
  while (C < 8 && slice(C) > two) C *= 2;
  if (slice(C) > one) C = 16;
  if (slice(C) > one) return false;
  while (C < 8 && rows * C < api_sm_count() && slice(C) >= 32768) C *= 2;
  sp.V = V;
  sp.C = C;
  sp.svec = static_cast<int32_t>((nvec + C - 1) / C);
  sp.gvec = static_cast<int32_t>(segment(C));
  sp.rvec = sp.gvec;
  sp.stages = 0;
  sp.H = 1;
  smem = row_bytes(sp.rvec, 0);
  return true;
}

// L2 that rows being read again may take.
constexpr int64_t kL2Rows = 96 << 20;

// The split of rows that fill the SMs' slots (two CTAs each): few CTAs per row,
// since a CTA's fixed costs and a cluster's waits then come less often; the row
// is streamed again in each pass.  `again`: as few as leave the rows in flight to
// L2; else as few as fill the slots.  extra(svec): a CTA's bytes beside its
// rings.  False: few rows, or no fewer CTAs than sp has; those are held whole.
template <typename Extra>
bool split_stream(int64_t rows, int32_t V, int32_t dtype, bool again, bool ring, int max_c,
                  Extra&& extra, RowSplit& sp, size_t& smem) {
  const int vw = 16 / elem_bytes(dtype);
  const int64_t nvec = (static_cast<int64_t>(V) + vw - 1) / vw;
  const int64_t slots = 2LL * api_sm_count();
  int C = 1;
  while (C < sp.C && ((again && slots / C * nvec * 16 > kL2Rows) || 5 * rows * C < 4 * slots)) C *= 2;
  if (C > max_c || C >= sp.C) return false;
  const int32_t svec = static_cast<int32_t>((nvec + C - 1) / C);
  const size_t work = extra(svec), room = kSmemSm / 2 - kSmemReserved;
  if (work > room) return false;
  const int64_t fits_too = static_cast<int64_t>(room - work) / row_bytes(1, 0);  // vectors per warp
  if (ring && fits_too < 2 * kStage) return false;
  sp.C = C;
  sp.svec = svec;
  sp.gvec = (svec + kRowWarps - 1) / kRowWarps;
  sp.rvec = ring ? 0 : std::min(sp.gvec, static_cast<int32_t>(fits_too) / kStage * kStage);
  sp.stages = ring ? std::min(kMaxRing, static_cast<int>(fits_too / kStage)) : 0;
  smem = row_bytes(sp.rvec, sp.stages);
  return true;
}

// What sampling's kernel is asked for, and the top logits.
enum FilterKind { kTokens, kFilteredAlone, kTopLogits };

// Their split; four histograms per CTA keep the part of a row small that a token is
// drawn from (2304 x 152064 fp32 top-p takes 1.36 times as long with one, 1.09 with
// two; 1024 x 128256 bf16 mixed 1.14, 1.05).
// Times of C = 1, of 2 and of rows held whole, by the first of them.  Sampling, whose
// first pass is its longest, takes the smallest C although rows in flight may overflow
// L2: 2304 x 152064 fp32 top-p 1, 1.12, 2.3; 320 rows 1, 1.17, 1.57; 1024 x 128256
// bf16 mixed 1, 1.04, 1.35.  So it does (us) where a second wave of CTAs is nearly empty
// (305 to 379 rows: tokens of 320 x 128256 bf16 101, held 117; of 320 x 50257 fp32
// 70, 107), but for filtered bf16 rows alone whose slices fill their shared memory
// to three quarters (320 x 128256 117, held 113, top-p alone 193, 166; 370 x 80000
// 130, 113; less full, 345 x 90000 93, 111, 345 x 175000 164, 209).  Top logits
// leave rows to L2: the 256 largest of 1024 x 152064 fp32 1.07, 1, 1.76; of 2048 x
// 152064 bf16 1, 1.39, 1.82; 100 of 333 x 50257 fp32 1, 1.28, 1.57.
bool split_filter(int64_t rows, int32_t V, int32_t dtype, FilterKind kind, RowSplit& sp, size_t& smem) {
  constexpr size_t fixed = (sizeof(FilterShared) + 127) / 128 * 128;
  const bool top = kind == kTopLogits;
  const int H = top ? 1 : kMaxH;
  if (!split_row(rows, V, dtype, fixed + work_bytes(1), sp, smem)) return false;
  const int64_t slots = 2LL * api_sm_count();
  const bool held = kind == kFilteredAlone && dtype == SPECV_BF16 && rows > slots && 4 * rows < 5 * slots &&
                    4 * smem >= 3 * (kSmemSm / 2 - kSmemReserved - fixed - work_bytes(1));
  const int max_c = !held && V / H <= kMaxBinned ? kMaxParts / H : 0;
  if (split_stream(rows, V, dtype, top, false, max_c, [&](int32_t) { return fixed + work_bytes(H); }, sp, smem)) sp.H = H;
  smem += work_bytes(sp.H);
  return true;
}

// 2^(63 + j/32).
BinTable make_table() {
  BinTable t;
  for (int j = 0; j < kGrid; ++j)
    t.e[j] = static_cast<uint64_t>(std::ldexp(std::exp2(static_cast<long double>(j) / kGrid), 63));
  return t;
}

specv_status launched(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return api_fail(SPECV_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
  return api_done(1);
}

}  // namespace

extern "C" {

specv_status specv_sample(const specv_sample_args* a, void* stream) {
  api_done(0);
  if (!a) return api_fail(SPECV_ERR_INVALID_ARG, "args is NULL");
  const int32_t B = a->B, R = a->R, V = a->V;
  specv_status st = check_rows("B", B, V, a->dtype);
  if (st != SPECV_OK) return st;
  if (R < 1) return api_fail(SPECV_ERR_INVALID_ARG, "R=%d < 1", R);
  if ((a->uniforms == nullptr) != (a->tokens == nullptr))
    return api_fail(SPECV_ERR_INVALID_ARG, "uniforms and tokens are given together");
  if (!a->tokens && !a->filtered) return api_fail(SPECV_ERR_INVALID_ARG, "neither tokens nor filtered is given");
  if (a->prob && !a->tokens) return api_fail(SPECV_ERR_INVALID_ARG, "prob needs tokens");
  if (B == 0) return api_done(0);
  if (!a->logits || !a->temperature) return api_fail(SPECV_ERR_INVALID_ARG, "a required pointer is NULL");
  const int es = elem_bytes(a->dtype);
  if (!aligned(a->logits, es) || !aligned(a->filtered, es) || !aligned(a->temperature, 4) || !aligned(a->top_k, 4) ||
      !aligned(a->top_p, 4) || !aligned(a->min_p, 4) || !aligned(a->uniforms, 4) || !aligned(a->tokens, 4) ||
      !aligned(a->prob, 4) || !aligned(a->kept, 4) || !aligned(a->row_status, 4))
    return api_fail(SPECV_ERR_INVALID_ARG, "a pointer is not aligned to its element size");
  if (a->row_stride < V || (a->filtered && a->filtered_row_stride < V))
    return api_fail(SPECV_ERR_INVALID_ARG, "row stride smaller than V");
  if (B > 1 && (a->batch_stride < (R - 1) * a->row_stride + V ||
                (a->filtered && a->filtered_batch_stride < (R - 1) * a->filtered_row_stride + V)))
    return api_fail(SPECV_ERR_INVALID_ARG, "batch stride too small for %d rows", R);
  const int64_t rows = static_cast<int64_t>(B) * R;
  FilterParams p = {};
  size_t smem;
  if (!split_filter(rows, V, a->dtype, a->tokens ? kTokens : kFilteredAlone, p.sp, smem))
    return api_fail(SPECV_ERR_UNSUPPORTED, "V=%d does not fit on chip", V);
  if (rows * p.sp.C > 0x7fffffffLL) return api_fail(SPECV_ERR_UNSUPPORTED, "B*R too large");
  p.rows = static_cast<int32_t>(rows);
  p.R = R;
  p.z = a->logits;
  p.bs = a->batch_stride;
  p.rs = a->row_stride;
  p.temp = a->temperature;
  p.top_k = a->top_k;
  p.top_p = a->top_p;
  p.min_p = a->min_p;
  p.u = a->uniforms;
  p.tokens = a->tokens;
  p.prob = a->prob;
  p.kept = a->kept;
  p.out = a->filtered;
  p.obs = a->filtered_batch_stride;
  p.ors = a->filtered_row_stride;
  p.status = a->row_status;
  static const BinTable table = make_table();
  p.tab = table;
  return launched(launch_sample_filter(a->dtype, smem, static_cast<cudaStream_t>(stream), p), "sample");
}

specv_status specv_top_logits(const specv_top_args* a, void* stream) {
  api_done(0);
  if (!a) return api_fail(SPECV_ERR_INVALID_ARG, "args is NULL");
  const int32_t B = a->B, V = a->V, k = a->k;
  specv_status st = check_rows("B", B, V, a->dtype);
  if (st != SPECV_OK) return st;
  if (k < 1 || k > SPECV_MAX_TOP) return api_fail(SPECV_ERR_INVALID_ARG, "k=%d outside [1, %d]", k, SPECV_MAX_TOP);
  if (!(a->temperature >= 1e-3f && a->temperature <= 1e3f))
    return api_fail(SPECV_ERR_INVALID_ARG, "temperature=%g outside [1e-3, 1e3]", static_cast<double>(a->temperature));
  if (B == 0) return api_done(0);
  if (!a->logits || !a->ids || !a->values) return api_fail(SPECV_ERR_INVALID_ARG, "a required pointer is NULL");
  const int es = elem_bytes(a->dtype);
  if (!aligned(a->logits, es) || !aligned(a->ids, 4) || !aligned(a->values, 4) || !aligned(a->lse, 4) ||
      !aligned(a->row_status, 4))
    return api_fail(SPECV_ERR_INVALID_ARG, "a pointer is not aligned to its element size");
  if (a->row_stride < V) return api_fail(SPECV_ERR_INVALID_ARG, "row stride smaller than V");
  TopParams p = {};
  size_t smem;
  if (!split_filter(B, V, a->dtype, kTopLogits, p.sp, smem))
    return api_fail(SPECV_ERR_UNSUPPORTED, "V=%d does not fit on chip", V);
  if (static_cast<int64_t>(B) * p.sp.C > 0x7fffffffLL) return api_fail(SPECV_ERR_UNSUPPORTED, "B too large");
  p.rows = B;
  p.k = k;
  p.z = a->logits;
  p.rs = a->row_stride;
  p.invT = 1.0 / static_cast<double>(a->temperature);
  p.c = static_cast<float>(1.4426950408889634 * p.invT);
  p.ids = a->ids;
  p.values = a->values;
  p.lse = a->lse;
  p.status = a->row_status;
  return launched(launch_top_logits(a->dtype, smem, static_cast<cudaStream_t>(stream), p), "top-logits");
}

}  // extern "C"

namespace {

specv_status check_distill(const specv_distill_args* a) {
  if (!a) return api_fail(SPECV_ERR_INVALID_ARG, "args is NULL");
  const int32_t N = a->N, V = a->V, K = a->K;
  specv_status st = check_rows("N", N, V, a->dtype);
  if (st != SPECV_OK) return st;
  if (K < 1 || K > SPECV_MAX_TOP) return api_fail(SPECV_ERR_INVALID_ARG, "K=%d outside [1, %d]", K, SPECV_MAX_TOP);
  if (!(a->temperature >= 1e-3f && a->temperature <= 1e3f))
    return api_fail(SPECV_ERR_INVALID_ARG, "temperature=%g outside [1e-3, 1e3]", static_cast<double>(a->temperature));
  if (a->flags & ~SPECV_DISTILL_TAIL) return api_fail(SPECV_ERR_INVALID_ARG, "unknown flags 0x%x", a->flags);
  if ((a->flags & SPECV_DISTILL_TAIL) && N > 0 && !a->teacher_lse)
    return api_fail(SPECV_ERR_INVALID_ARG, "SPECV_DISTILL_TAIL needs teacher_lse");
  if (N == 0) return SPECV_OK;
  if (!a->logits || !a->teacher_ids || !a->teacher_logits)
    return api_fail(SPECV_ERR_INVALID_ARG, "a required pointer is NULL");
  const int es = elem_bytes(a->dtype);
  if (!aligned(a->logits, es) || !aligned(a->grad, es) || !aligned(a->teacher_ids, 4) || !aligned(a->teacher_logits, 4) ||
      !aligned(a->teacher_lse, 4) || !aligned(a->weights, 4) || !aligned(a->loss, 4) || !aligned(a->grad_loss, 4) ||
      !aligned(a->row_status, 4))
    return api_fail(SPECV_ERR_INVALID_ARG, "a pointer is not aligned to its element size");
  if (!aligned(a->stats, 16)) return api_fail(SPECV_ERR_INVALID_ARG, "stats is not 16-byte aligned");
  if (a->row_stride < V || (a->grad && a->grad_row_stride < V))
    return api_fail(SPECV_ERR_INVALID_ARG, "row stride smaller than V");
  if (a->teacher_stride < K) return api_fail(SPECV_ERR_INVALID_ARG, "teacher_stride smaller than K");
  return SPECV_OK;
}

// The split of rows that are held, and with it the widest row that is taken.
// (a held row's bits are at most a 16th of its bytes)
bool split_distill(const specv_distill_args* a, RowSplit& sp, size_t& smem) {
  const int vw = 16 / elem_bytes(a->dtype);
  const size_t entries = static_cast<size_t>(a->K) * 20;
  const size_t bits = distill_bytes(static_cast<int32_t>((static_cast<int64_t>(a->V) + vw - 1) / vw), vw, 0);
  return split_row(a->N, a->V, a->dtype, kDistillStatic + std::min<size_t>(bits, 16384) + entries, sp, smem);
}

DistillParams distill_params(const specv_distill_args* a) {
  DistillParams p = {};
  p.N = a->N;
  p.K = a->K;
  p.z = a->logits;
  p.rs = a->row_stride;
  p.ids = a->teacher_ids;
  p.tl = a->teacher_logits;
  p.ts = a->teacher_stride;
  p.tlse = a->teacher_lse;
  p.weight = a->weights;
  const double inv = 1.0 / static_cast<double>(a->temperature);
  p.ih = static_cast<float>(inv);
  p.il = static_cast<float>(inv - static_cast<double>(p.ih));
  p.c = static_cast<float>(1.4426950408889634 * inv);
  p.tail = (a->flags & SPECV_DISTILL_TAIL) != 0;
  p.stats = reinterpret_cast<float4*>(a->stats);
  p.grad = a->grad;
  p.grs = a->grad_row_stride;
  p.sp.V = a->V;
  return p;
}

}  // namespace

extern "C" {

specv_status specv_distill(const specv_distill_args* a, void* stream) {
  api_done(0);
  specv_status st = check_distill(a);
  if (st != SPECV_OK) return st;
  if (a->N == 0) return api_done(0);
  if (!a->loss) return api_fail(SPECV_ERR_INVALID_ARG, "a required pointer is NULL");
  if (a->grad_loss) return api_fail(SPECV_ERR_INVALID_ARG, "grad_loss belongs to specv_distill_backward");
  DistillParams p = distill_params(a);
  size_t smem;
  const int vw = 16 / elem_bytes(a->dtype);
  if (!split_distill(a, p.sp, smem))
    return api_fail(SPECV_ERR_UNSUPPORTED, "V=%d does not fit on chip", a->V);
  // (With a gradient the rows are read again: by one CTA each, in the place of as few
  // as leave them to L2, 1024 x 152064 fp32 take 10 % longer, 300 rows 18 %.)
  split_stream(a->N, a->V, a->dtype, a->grad != nullptr, true, kMaxCluster,
               [&](int32_t svec) { return kDistillStatic + distill_bytes(svec, vw, a->K); }, p.sp, smem);
  smem += distill_bytes(p.sp.svec, vw, a->K);
  if (static_cast<int64_t>(a->N) * p.sp.C > 0x7fffffffLL) return api_fail(SPECV_ERR_UNSUPPORTED, "N too large");
  p.loss = a->loss;
  p.status = a->row_status;
  p.stall[0] = api_test_stall('C');
  p.stall[1] = api_test_stall('D');
  return launched(launch_distill(a->dtype, smem, static_cast<cudaStream_t>(stream), p), "distill");
}

specv_status specv_distill_backward(const specv_distill_args* a, void* stream) {
  api_done(0);
  specv_status st = check_distill(a);
  if (st != SPECV_OK) return st;
  if (a->N == 0) return api_done(0);
  if (!a->stats || !a->grad) return api_fail(SPECV_ERR_INVALID_ARG, "a required pointer is NULL");
  RowSplit held;
  size_t smem;
  if (!split_distill(a, held, smem))  // (no statistics come of such rows, and the kernel's indices hold no others)
    return api_fail(SPECV_ERR_UNSUPPORTED, "V=%d does not fit on chip", a->V);
  if (static_cast<int64_t>(a->N) * ((a->V + 6) / back_piece(16 / elem_bytes(a->dtype)) + 1) > 0x7fffffffLL)
    return api_fail(SPECV_ERR_UNSUPPORTED, "N too large");
  DistillParams p = distill_params(a);
  p.gloss = a->grad_loss;
  return launched(launch_distill_backward(a->dtype, static_cast<cudaStream_t>(stream), p), "distill-backward");
}

}  // extern "C"
