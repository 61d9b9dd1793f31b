// C ABI of the orthogonalised update: argument checks, the workspace, bounds on the
// singular values, and the launches on the caller's stream.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "api.cuh"
#include "orth_launch.cuh"
#include "product_launch.cuh"

using namespace specv;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int64_t up_to(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

constexpr int kMostSteps = kSmallSteps;
constexpr double kMostGrowth = 1024;

// The largest |a x + b x^3 + c x^5| for x in [0, r], and |b t + c t^2| for t in [0, r^2].
double step_bound(double a, double b, double c, double r) {
  auto f = [&](double t) { return std::fabs(std::sqrt(t) * (a + t * (b + t * c))); };
  double most = f(r * r);
  const double A = 5 * c, B = 3 * b, C = a, disc = B * B - 4 * A * C;
  for (double t : {A != 0 && disc >= 0 ? (-B + std::sqrt(disc)) / (2 * A) : -1.0,
                   A != 0 && disc >= 0 ? (-B - std::sqrt(disc)) / (2 * A) : -1.0, A == 0 && B != 0 ? -C / B : -1.0})
    if (t > 0 && t < r * r) most = std::max(most, f(t));
  return most;
}
double poly_bound(double b, double c, double r) {
  auto g = [&](double t) { return std::fabs(t * (b + t * c)); };
  double most = g(r * r);
  const double t = c != 0 ? -b / (2 * c) : -1.0;
  if (t > 0 && t < r * r) most = std::max(most, g(t));
  return most;
}
// The power of two by which a matrix of entries up to `most` is kept in fp16 (up to 32768,
// half of its range: the bounds hold for exact steps).
double keep_scale(double most) { return std::exp2(std::floor(std::log2(32768.0 / std::max(most, 1e-30)))); }

// CTAs of a cluster that holds a matrix of a smaller side up to 128 in its shared memory
// (powers of two up to 16, so that they share its rows evenly), or 0: it does not fit.
int small_ctas(int32_t s, int32_t t) {
  if (s > kSmallSide || t > 16 * kSmallSide) return 0;
  int C = 1;
  while (C * kSmallSide < t) C *= 2;
  return C;
}

// How a product is cut: into tiles of 128 x 128, a CTA each (half), or of 256 x 256, a pair
// each, and K into parts whose sums a pass of its own joins; whatever ends soonest.  Cycles of
// a block of K: 256 and 512 are the tensor core's, the more SMs take part the more are L2's
// (up to 540 and 620); and of what is not hidden under the next tile, about 4000 and 6000.
// The join: a launch, and the sums' bytes.  us of a call by 128, by 256 and by the better of
// the two: 1000 x 2333 205, 240, 205; 1024 x 4096 257, 261, 242; 24 x 1024 x 1024 830, 687,
// 687; 4096 x 4096 1611, 1040, 1040.  With and without parts of K: 100 x 9000 239, 831;
// 250 x 16384 297, 1347; 8192 x 500 225, 425; 8192 x 2048 600, 632.
struct Cut {
  bool half;
  int32_t splits;
};

Cut product_cut(ProductParams p, bool parts) {
  const int64_t blocks = (p.K + kProdBK - 1) / kProdBK * (p.fine ? 3 : 1);
  Cut best = {};
  double least = 1e30;
  for (bool half : {false, true}) {
    const int64_t ctas = half ? api_sm_count() : api_sm_count() / 2;
    p.splits = 1;
    const int64_t tiles = product_units(p, half ? kProdHalf : kProdTile);
    for (int64_t splits = 1; splits == 1 || (parts && splits <= 64 && splits * tiles <= 2 * ctas && splits * 8 <= blocks); ++splits) {
      const int64_t units = tiles * splits, rounds = (units + ctas - 1) / ctas, part = (blocks + splits - 1) / splits;
      const double busy = std::min(1.0, static_cast<double>(units) / ctas);
      double cycles = half ? rounds * part * (280 + 260 * busy) + 4000 : rounds * part * (540 + 80 * busy) + 6000;
      if (splits > 1) cycles += 9000 + 4.0 * p.batch * p.M * p.N * (splits + 1) / 4000;
      if (cycles < least) least = cycles, best = {half, static_cast<int32_t>(splits)};
    }
  }
  return best;
}

struct OrthSpace {
  size_t part, hi[2], lo[2], gram[2], poly[2], sums, bytes;  // (of S and P: fp16, and what that leaves out)
  int64_t ld, lds;  // strides of X, of S and P
  int32_t s, t, blocks;
  bool tall, fine;
  Cut gram_cut;
};

OrthSpace orth_space(int32_t B, int32_t m, int32_t n) {
  OrthSpace w = {};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  w.tall = m > n;
  w.s = std::min(m, n), w.t = std::max(m, n);
  w.ld = up_to(n, 8), w.lds = up_to(w.s, 8);
  // blocks of the passes over G: 8 vectors a thread, or four blocks an SM over the batch
  const int64_t vectors = static_cast<int64_t>(m) * ((n + 3) / 4);
  w.blocks = static_cast<int32_t>(std::max<int64_t>(
      1, std::min((vectors + 8 * kOrthThreads - 1) / (8 * kOrthThreads), std::max<int64_t>(1, 4LL * api_sm_count() / B))));
  if (small_ctas(w.s, w.t)) return w;  // (in one kernel, on chip)
  w.part = take(sizeof(ScaledSquares) * static_cast<size_t>(B) * w.blocks);
  const size_t x = 2 * static_cast<size_t>(B) * m * w.ld, q = 2 * static_cast<size_t>(B) * w.s * w.lds;
  w.hi[0] = take(x), w.hi[1] = take(x), w.lo[0] = take(x);
  w.fine = w.s <= kProdTile;
  // (what X's fp16 leaves out is read and written by the same epilogue alone, unless products read it)
  w.lo[1] = w.fine ? take(x) : w.lo[0];
  for (int k = 0; k <= w.fine; ++k) w.gram[k] = take(q), w.poly[k] = take(q);
  ProductParams p = {};
  p.M = p.N = w.s, p.K = w.t, p.batch = B, p.symmetric = 1, p.fine = w.fine;
  w.gram_cut = product_cut(p, true);
  if (w.gram_cut.splits > 1) w.sums = take(2 * q * w.gram_cut.splits);
  w.bytes = at;
  return w;
}

specv_status check_orth(const specv_orth_args* a) {
  if (!a) return api_fail(SPECV_ERR_INVALID_ARG, "args is NULL");
  if (a->B < 0) return api_fail(SPECV_ERR_INVALID_ARG, "B=%d < 0", a->B);
  if (a->m < 1 || a->n < 1) return api_fail(SPECV_ERR_INVALID_ARG, "m=%d, n=%d: less than 1", a->m, a->n);
  if (a->dtype != SPECV_BF16 && a->dtype != SPECV_FP32)
    return api_fail(SPECV_ERR_INVALID_ARG, "dtype=%d is not SPECV_BF16 or SPECV_FP32", a->dtype);
  if (a->steps < 1 || a->steps > kMostSteps)
    return api_fail(SPECV_ERR_INVALID_ARG, "steps=%d outside [1, %d]", a->steps, kMostSteps);
  if (!std::isfinite(a->a) || !std::isfinite(a->b) || !std::isfinite(a->c))
    return api_fail(SPECV_ERR_INVALID_ARG, "a coefficient is not finite");
  double r = 1;
  for (int k = 0; k < a->steps; ++k) {
    r = 1.01 * step_bound(a->a, a->b, a->c, r);
    if (!(r <= kMostGrowth))
      return api_fail(SPECV_ERR_INVALID_ARG, "coefficients (%g, %g, %g) may let singular values grow past %g in %d steps",
                      static_cast<double>(a->a), static_cast<double>(a->b), static_cast<double>(a->c), kMostGrowth, a->steps);
  }
  if (std::max(a->m, a->n) > kProdMost)
    return api_fail(SPECV_ERR_UNSUPPORTED, "m=%d, n=%d: more than %d", a->m, a->n, kProdMost);
  if (a->B == 0) return SPECV_OK;
  if (!a->update || !a->out) return api_fail(SPECV_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned(a->update, a->dtype == SPECV_BF16 ? 2 : 4) || !aligned(a->out, 2) || !aligned(a->norm, 4) ||
      !aligned(a->row_status, 4))
    return api_fail(SPECV_ERR_INVALID_ARG, "a pointer is not aligned to its element size");
  if (a->m > 1 && (a->row_stride < a->n || a->out_row_stride < a->n))
    return api_fail(SPECV_ERR_INVALID_ARG, "row stride smaller than n");
  if (a->B > 1 && (a->batch_stride < (a->m - 1) * a->row_stride + a->n ||
                   a->out_batch_stride < (a->m - 1) * a->out_row_stride + a->n))
    return api_fail(SPECV_ERR_INVALID_ARG, "batch stride too small for %d rows", a->m);
  const int64_t tiles = up_to(a->m, kProdTile) / kProdTile * (up_to(a->n, kProdTile) / kProdTile);
  if (tiles * a->B > (1 << 30) || a->B > 65535) return api_fail(SPECV_ERR_UNSUPPORTED, "B, m and n too large");
  return SPECV_OK;
}

#define TRY(x)                       \
  do {                               \
    const specv_status st_ = (x);    \
    if (st_ != SPECV_OK) return st_; \
  } while (0)

struct OrthRun {
  const specv_orth_args* a;
  OrthSpace w;
  uint8_t* ws;
  cudaStream_t s;
  int launches = 0;

  uint16_t* at(size_t off) const { return reinterpret_cast<uint16_t*>(ws + off); }
  specv_status done(cudaError_t e, const char* what) {
    if (e != cudaSuccess) return api_fail(SPECV_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    ++launches;
    return SPECV_OK;
  }
  // half: tiles of 128 x 128 by one CTA each.
  ProductParams product(int32_t M, int32_t N, int32_t K, bool symmetric, bool& half) const {
    ProductParams p = {};
    p.M = M, p.N = N, p.K = K, p.batch = a->B, p.splits = 1;
    p.symmetric = symmetric, p.fine = w.fine;
    half = product_cut(p, false).half;
    p.status = a->row_status, p.status_n = a->B;
    return p;
  }
  int64_t zx() const { return a->m * w.ld; }
  int64_t zs() const { return w.s * w.lds; }
  specv_status x_map(CUtensorMap* m, bool mn, size_t off) const {
    return operand_map(m, false, mn, at(off), a->n, a->m, a->B, w.ld, zx());
  }
  specv_status s_map(CUtensorMap* m, size_t off) const {
    return operand_map(m, false, false, at(off), w.s, w.s, a->B, w.lds, zs());
  }
  specv_status box_map(CUtensorMap* m, size_t off, int64_t cols, int64_t rows, int64_t ld, int width = 64) const {
    return product_map(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, at(off), cols, rows, a->B, 2 * ld, 2 * rows * ld, 32, width);
  }

  // S, then P = b S + c S S
  template <bool FINE>
  specv_status symmetric(int from, const SmallStep& f) {
    const bool first = launches == 2;  // (the test hooks')
    bool half;
    {
      ProductParams p = product(w.s, w.s, w.t, true, half);
      half = w.gram_cut.half;
      p.splits = w.gram_cut.splits;
      TRY(x_map(&p.a, w.tall, w.hi[from]));
      if (FINE) TRY(x_map(&p.a_low, w.tall, w.lo[from]));
      p.b = p.a, p.b_low = p.a_low;
      if (first) p.stall = api_test_stall('F');
      if (p.splits > 1) {
        SumEpi::Params e = {};
        TRY(product_map(&e.out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, at(w.sums), w.s, w.s, a->B * p.splits, 4 * w.lds, 4 * zs(), 32));
        e.cols = w.s, e.splits = p.splits;
        TRY(done(launch_orth_sums(half, w.tall, p, e, s), "orthogonalize-gram"));
        OrthJoinParams j = {};
        j.n = w.s, j.splits = p.splits, j.patches = (w.s + 63) / 64, j.sum = reinterpret_cast<const float*>(at(w.sums));
        j.hi = at(w.gram[0]), j.lo = FINE ? at(w.gram[1]) : nullptr, j.ld = w.lds, j.alpha = f.gram;
        TRY(done(launch_orth_join(j, a->B, s), "orthogonalize-join"));
      } else {
        typename SymEpi<false, FINE>::Params e = {};
        TRY(sym_out(e, w.gram, FINE));
        e.alpha = f.gram;
        TRY(done(launch_orth_gram<FINE>(half, w.tall, p, e, s), "orthogonalize-gram"));
      }
    }
    ProductParams p = product(w.s, w.s, w.s, true, half);
    TRY(s_map(&p.a, w.gram[0]));
    if (FINE) TRY(s_map(&p.a_low, w.gram[1]));
    p.b = p.a, p.b_low = p.a_low;
    typename SymEpi<true, FINE>::Params e = {};
    TRY(sym_out(e, w.poly, FINE));
    TRY(box_map(&e.chi, w.gram[0], w.s, w.s, w.lds));
    if (FINE) TRY(box_map(&e.clo, w.gram[1], w.s, w.s, w.lds));
    e.alpha = f.poly, e.beta = f.poly_s;
    if (first) p.stall_read = api_test_stall('J');
    return done(launch_orth_poly<FINE>(half, p, e, s), "orthogonalize-poly");
  }
  template <typename Params>
  specv_status sym_out(Params& e, const size_t (&to)[2], bool fine) const {
    TRY(box_map(&e.hi, to[0], w.s, w.s, w.lds));
    TRY(box_map(&e.mirror_hi, to[0], w.s, w.s, w.lds, 0));
    if (fine) TRY(box_map(&e.lo, to[1], w.s, w.s, w.lds));
    if (fine) TRY(box_map(&e.mirror_lo, to[1], w.s, w.s, w.lds, 0));
    e.n = w.s;
    return SPECV_OK;
  }

  // The factors that a step multiplies its products by: what they are kept times, before and after.
  SmallStep factors(double r, double sx, double sn) const {
    const double ss = keep_scale(r * r), sp = keep_scale(poly_bound(a->b, a->c, r));
    return {static_cast<float>(ss / (sx * sx)), static_cast<float>(a->c * sp / (ss * ss)), static_cast<float>(a->b * sp / ss),
            static_cast<float>(sn / (sp * sx)), static_cast<float>(a->a * sn / sx)};
  }

  specv_status small() {
    SmallParams p = {};
    p.s = w.s, p.t = w.t, p.tall = w.tall, p.steps = a->steps;
    p.in = a->update, p.row_stride = a->m > 1 ? a->row_stride : a->n, p.batch_stride = a->B > 1 ? a->batch_stride : 0;
    p.out = static_cast<uint16_t*>(a->out);
    p.out_row_stride = a->m > 1 ? a->out_row_stride : a->n, p.out_batch_stride = a->B > 1 ? a->out_batch_stride : 0;
    p.vec = aligned(a->update, a->dtype == SPECV_BF16 ? 8 : 16) && p.row_stride % 4 == 0 && p.batch_stride % 4 == 0;
    p.out_vec = aligned(a->out, 8) && p.out_row_stride % 4 == 0 && p.out_batch_stride % 4 == 0;
    p.norm = a->norm, p.status = a->row_status;
    double r = 1, sx = keep_scale(r);
    p.scale = static_cast<float>(sx);
    p.stall = api_test_stall('K');
    for (int k = 0; k < a->steps; ++k) {
      const double next = 1.01 * step_bound(a->a, a->b, a->c, r), sn = k + 1 == a->steps ? 1.0 : keep_scale(next);
      p.step[k] = factors(r, sx, sn);
      r = next, sx = sn;
    }
    return done(launch_orth_small(a->dtype, p, small_ctas(w.s, w.t), a->B, s), "orthogonalize");
  }

  specv_status all() {
    if (small_ctas(w.s, w.t)) return small();
    double r = 1, sx = keep_scale(r);
    {
      OrthInParams p = {};
      p.rows = a->m, p.cols = a->n, p.batch = a->B, p.blocks = w.blocks;
      p.in = a->update, p.row_stride = a->m > 1 ? a->row_stride : a->n, p.batch_stride = a->B > 1 ? a->batch_stride : 0;
      const int vw = a->dtype == SPECV_BF16 ? 8 : 4;
      p.vec = aligned(a->update, 16) && p.row_stride % vw == 0 && p.batch_stride % vw == 0;
      p.part = reinterpret_cast<ScaledSquares*>(ws + w.part);
      p.hi = at(w.hi[0]), p.lo = at(w.lo[0]), p.ld = w.ld, p.matrix = zx(), p.scale = static_cast<float>(sx);
      p.norm = a->norm, p.status = a->row_status;
      if (p.row_stride == a->n && w.ld == a->n) p.cols *= p.rows, p.ld = p.cols, p.rows = 1;
      TRY(done(launch_orth_squares(a->dtype, p, s), "orthogonalize-norm"));
      TRY(done(launch_orth_scale(a->dtype, p, s), "orthogonalize-scale"));
    }
    for (int k = 0; k < a->steps; ++k) {
      const int from = k & 1;
      const bool last = k + 1 == a->steps;
      const double next = 1.01 * step_bound(a->a, a->b, a->c, r), sn = last ? 1.0 : keep_scale(next);
      const SmallStep f = factors(r, sx, sn);
      TRY(w.fine ? symmetric<true>(from, f) : symmetric<false>(from, f));
      // X' = a X + P X, or a X + X P (P is its own transpose)
      bool half;
      ProductParams p = product(a->m, a->n, w.s, false, half);
      if (k == 0) p.stall_read = api_test_stall('J');
      TRY(s_map(w.tall ? &p.b : &p.a, w.poly[0]));
      TRY(x_map(w.tall ? &p.a : &p.b, !w.tall, w.hi[from]));
      if (w.fine) {
        TRY(s_map(w.tall ? &p.b_low : &p.a_low, w.poly[1]));
        TRY(x_map(w.tall ? &p.a_low : &p.b_low, !w.tall, w.lo[from]));
      }
      auto step = [&](auto& e) {
        TRY(box_map(&e.xhi, w.hi[from], a->n, a->m, w.ld));
        TRY(box_map(&e.xlo, w.lo[from], a->n, a->m, w.ld));
        e.rows = a->m, e.cols = a->n;
        e.alpha = f.step, e.beta = f.step_y;
        return SPECV_OK;
      };
      if (!last) {
        StepEpi<false>::Params e = {};
        TRY(step(e));
        TRY(box_map(&e.hi, w.hi[from ^ 1], a->n, a->m, w.ld));
        TRY(box_map(&e.lo, w.lo[from ^ 1], a->n, a->m, w.ld));
        TRY(done(launch_orth_step(half, !w.tall, p, e, s), "orthogonalize-step"));
      } else {
        StepEpi<true>::Params e = {};
        TRY(step(e));
        const int64_t rs = a->m > 1 ? a->out_row_stride : up_to(a->n, 8), bs = a->B > 1 ? a->out_batch_stride : 0;
        e.stride = rs, e.zstride = bs;
        // (TMA stores whole 16-byte words: what lies behind a row stays as it is)
        if (aligned(a->out, 16) && rs % 8 == 0 && bs % 8 == 0 && a->n % 8 == 0)
          TRY(product_map(&e.hi, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a->out, a->n, a->m, a->B, 2 * rs, 2 * bs, 32, 64));
        else
          e.direct = static_cast<uint16_t*>(a->out);
        TRY(done(launch_orth_last(half, !w.tall, p, e, s), "orthogonalize-last"));
      }
      r = next, sx = sn;
    }
    return SPECV_OK;
  }
};

}  // namespace

extern "C" {

size_t specv_orthogonalize_workspace_bytes(int32_t B, int32_t m, int32_t n) {
  if (B < 1 || m < 1 || n < 1) return 0;
  return orth_space(B, m, n).bytes;
}

specv_status specv_orthogonalize(const specv_orth_args* a, void* workspace, size_t workspace_bytes, void* stream) {
  api_done(0);
  TRY(check_orth(a));
  if (a->B == 0) return api_done(0);
  OrthRun run = {a, orth_space(a->B, a->m, a->n), static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream)};
  if (run.w.bytes && (!workspace || workspace_bytes < run.w.bytes))
    return api_fail(SPECV_ERR_WORKSPACE, "workspace of %zu bytes needed, got %zu", run.w.bytes, workspace ? workspace_bytes : 0);
  if (!aligned(workspace, 256)) return api_fail(SPECV_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
  TRY(run.all());
  return api_done(run.launches);
}

}  // extern "C"
