// C ABI of the cross entropy from hidden states: argument checks, the workspace, and the
// launches on the caller's stream.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "api.cuh"
#include "head_launch.cuh"
#include "product_launch.cuh"

using namespace specv;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int64_t up_to(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Rows beyond one tile are gathered, so that rows without weight cost nothing; fewer rows
// take the same tile whatever their number.
bool gathers(int32_t N) { return N > kProdTile; }

// Up to 128 rows go by tiles of 128 x 128, a CTA each: a pair's 256 rows cost the tensor core
// twice the time for the same bytes of the head, nearly what those take from HBM (45 x 4096 x
// 128256: 182 us by pairs, 176, both with sums in chunks of 8 blocks).
bool few_rows(int32_t N) { return N <= kProdHalf; }

// A call that computes the loss and the gradients keeps the logits' weights in fp16 where
// they take no more than 1 GB (4096 rows of 131072 tokens), and computes the logits once:
// 6 N D V operations for 8.  Otherwise, and in a backward pass, the vocabulary is taken in
// pieces and the logits are computed again.  The limit is on the memory that a call asks for,
// not the faster side: 4096 x 4096 tokens of 131072 take 8.7 ms, of 152064 12.4 (1.52 and 1.23
// PFLOP/s of 6 N D V), all rows in use.
constexpr int64_t kKeepBytes = 1LL << 30;

// Tokens per piece of the vocabulary: dz of a piece takes 256 MB at most (pieces of equal
// size, of whole tiles).
int64_t piece_tokens(int32_t N, int32_t V, bool keep) {
  if (keep && 2 * up_to(N, kProdBK) * up_to(V, kProdTile) <= kKeepBytes) return up_to(V, kProdTile);
  const int64_t most = std::max<int64_t>((256LL << 20) / (2 * up_to(N, kProdBK)) / kProdTile * kProdTile, kProdTile);
  const int64_t pieces = (V + most - 1) / most;
  return up_to((V + pieces - 1) / pieces, kProdTile);
}

// Parts that K (a piece's tokens) is cut into for dh, whose tiles alone are few.  Tiles for
// every pair of SMs (or SM): eight units for each, so that a last round that is not full costs
// little (4096 x 4096 of 128256 tokens, 0.7 of the rows in use: 192 tiles on 76 pairs), in
// parts of 64 blocks at least.  Fewer: one unit for each, of 8 blocks at least.
int hidden_splits(int32_t N, int32_t D, int64_t tokens) {
  const int size = few_rows(N) ? kProdHalf : kProdTile;
  const int64_t tiles = up_to(N, size) / size * (up_to(D, size) / size);
  const int64_t groups = few_rows(N) ? api_sm_count() : api_sm_count() / 2, blocks = up_to(tokens, kProdBK) / kProdBK;
  const int64_t n = tiles >= groups ? std::min((8 * groups + tiles - 1) / tiles, blocks / 64) : std::min(groups / tiles, blocks / 8);
  return static_cast<int>(std::max<int64_t>(n, 1));
}

// Offsets of the workspace's parts (bytes; all multiples of 256).
struct HeadSpace {
  size_t count, most, late, err, place, source, target, row, bad, z_target, part, hidden, head, dz, sum, bytes;
  int64_t rows, ld, Dp, Ds, tokens;  // rows: N up to a block; ld: of part; Dp, Ds: strides of gathered rows and sums
  int splits;
  int part_cols;  // tokens per partial sum
  bool gather, copy_hidden, copy_head, grads, keep, half;
};

// keep: of a call that computes the loss too.
HeadSpace head_space(const specv_head_args* a, bool keep) {
  HeadSpace w = {};
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += (n + 255) / 256 * 256;
    return here;
  };
  const int64_t N = a->N, V = a->V, D = a->D;
  w.grads = a->grad_hidden || a->grad_head;
  w.rows = up_to(N, kProdBK);
  w.ld = up_to(N, 32);
  w.Dp = up_to(D, 8);
  w.Ds = up_to(D, 8);
  w.gather = gathers(a->N);
  const bool fits = aligned(a->hidden, 16) && (N <= 1 || a->hidden_stride % 8 == 0);
  w.copy_hidden = w.gather || w.grads || !fits;
  w.copy_head = !(aligned(a->head, 16) && (V <= 1 || a->head_stride % 8 == 0));
  w.count = take(4);
  w.most = take(4);
  w.late = take(4);
  w.err = take(4 * 1024);
  w.place = take(4 * N);
  w.source = take(4 * N);
  w.target = take(4 * N);
  w.row = take(sizeof(HeadRow) * N);
  w.bad = take(4 * N);
  w.z_target = take(4 * N);
  w.half = few_rows(a->N);
  w.part_cols = w.half ? kProdHalf / 2 : kProdTile / 2;
  w.part = take(sizeof(float2) * static_cast<size_t>((V + w.part_cols - 1) / w.part_cols) * w.ld);
  if (w.copy_hidden) w.hidden = take(2 * w.rows * w.Dp);
  if (w.copy_head) w.head = take(2 * static_cast<size_t>(V) * w.Dp);
  if (w.grads) {
    w.tokens = piece_tokens(a->N, a->V, keep);
    w.keep = keep && w.tokens >= a->V;
    w.dz = take(2 * static_cast<size_t>(w.rows) * w.tokens);
    if (a->grad_hidden) {
      w.splits = hidden_splits(a->N, a->D, w.tokens);
      w.sum = take(4 * static_cast<size_t>(w.splits) * w.rows * w.Ds);
    }
  }
  w.bytes = at;
  return w;
}

specv_status check_head(const specv_head_args* a) {
  if (!a) return api_fail(SPECV_ERR_INVALID_ARG, "args is NULL");
  if (a->N < 0) return api_fail(SPECV_ERR_INVALID_ARG, "N=%d < 0", a->N);
  if (a->V < 1) return api_fail(SPECV_ERR_INVALID_ARG, "V=%d < 1", a->V);
  if (a->D < 1) return api_fail(SPECV_ERR_INVALID_ARG, "D=%d < 1", a->D);
  if (a->dtype != SPECV_BF16 && a->dtype != SPECV_FP32)
    return api_fail(SPECV_ERR_INVALID_ARG, "dtype=%d is not SPECV_BF16 or SPECV_FP32", a->dtype);
  if (a->dtype != SPECV_BF16) return api_fail(SPECV_ERR_UNSUPPORTED, "hidden states and head are bf16");
  if (!(a->scale >= 1e-6f && a->scale <= 1e6f))
    return api_fail(SPECV_ERR_INVALID_ARG, "scale=%g outside [1e-6, 1e6]", static_cast<double>(a->scale));
  if (a->flags & ~SPECV_HEAD_TARGETS_ONLY) return api_fail(SPECV_ERR_INVALID_ARG, "unknown flags 0x%x", a->flags);
  if (std::max({a->N, a->V, a->D}) > kProdMost)
    return api_fail(SPECV_ERR_UNSUPPORTED, "N=%d, V=%d, D=%d: more than %d", a->N, a->V, a->D, kProdMost);
  if (a->N == 0 && !a->grad_head) return SPECV_OK;
  if (a->N > 0 && (!a->hidden || !a->targets)) return api_fail(SPECV_ERR_INVALID_ARG, "a required pointer is NULL");
  if (a->N > 0 && !a->head) return api_fail(SPECV_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned(a->hidden, 2) || !aligned(a->head, 2) || !aligned(a->grad_hidden, 2) || !aligned(a->grad_head, 2) ||
      !aligned(a->targets, 4) || !aligned(a->weights, 4) || !aligned(a->loss, 4) || !aligned(a->stats, 4) ||
      !aligned(a->grad_loss, 4) || !aligned(a->row_status, 4))
    return api_fail(SPECV_ERR_INVALID_ARG, "a pointer is not aligned to its element size");
  if ((a->N > 1 && a->hidden_stride < a->D) || (a->V > 1 && a->head_stride < a->D) ||
      (a->grad_hidden && a->N > 1 && a->grad_hidden_stride < a->D) ||
      (a->grad_head && a->V > 1 && a->grad_head_stride < a->D))
    return api_fail(SPECV_ERR_INVALID_ARG, "row stride smaller than D");
  return SPECV_OK;
}

#define TRY(x)                            \
  do {                                    \
    const specv_status st_ = (x);         \
    if (st_ != SPECV_OK) return st_;      \
  } while (0)

// The call's launches, counted; the first error ends it.
struct HeadRun {
  const specv_head_args* a;
  HeadSpace w;
  uint8_t* ws;
  cudaStream_t s;
  int launches = 0;

  template <typename T>
  T* at(size_t off) const {
    return reinterpret_cast<T*>(ws + off);
  }
  specv_status done(cudaError_t e, const char* what) {
    if (e != cudaSuccess) return api_fail(SPECV_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    ++launches;
    return SPECV_OK;
  }
  const uint16_t* hidden() const {
    return w.copy_hidden ? at<uint16_t>(w.hidden) : static_cast<const uint16_t*>(a->hidden);
  }
  int64_t hidden_stride() const { return w.copy_hidden ? w.Dp : a->N > 1 ? a->hidden_stride : up_to(a->D, 8); }
  const uint16_t* head() const { return w.copy_head ? at<uint16_t>(w.head) : static_cast<const uint16_t*>(a->head); }
  int64_t head_stride() const { return w.copy_head ? w.Dp : a->V > 1 ? a->head_stride : up_to(a->D, 8); }

  // Whether rows without a target have statistics.
  bool every_row() const { return !w.grads && !(a->flags & SPECV_HEAD_TARGETS_ONLY); }

  // Rows in use, and copies of operands that TMA cannot read in place.
  specv_status rows(bool backward) {
    HeadRowsParams r = {};
    r.N = a->N, r.V = a->V;
    r.target = a->targets, r.weight = a->weights, r.scale = a->scale, r.all = !backward && every_row();
    if (w.gather || w.grads) r.most = at<float>(w.most);
    if (backward) r.up = a->grad_loss, r.stats = a->stats, r.row = at<HeadRow>(w.row);
    if (w.gather) {
      r.count = at<int32_t>(w.count);
      r.place = at<int32_t>(w.place), r.source = at<int32_t>(w.source), r.use_target = at<int32_t>(w.target);
      TRY(done(launch_head_rows(r, s), "head-rows"));
    }
    if (w.copy_hidden) {
      HeadGatherParams p = {};
      p.N = a->N, p.D = a->D, p.pad_to = kProdBK;
      p.vec = aligned(a->hidden, 16) && (a->N <= 1 || a->hidden_stride % 8 == 0);
      if (w.gather) p.count = r.count, p.source = r.source;
      else p.info = r;
      if (w.grads) p.bad = at<int32_t>(w.bad), p.late = at<int32_t>(w.late);
      if (backward) {
        p.stats = a->stats, p.target = r.use_target, p.row = at<HeadRow>(w.row);
        p.head = static_cast<const uint16_t*>(a->head), p.head_stride = a->V > 1 ? a->head_stride : a->D;
      }
      p.in = static_cast<const uint16_t*>(a->hidden), p.in_stride = a->N > 1 ? a->hidden_stride : a->D;
      p.out = at<uint16_t>(w.hidden), p.out_stride = w.Dp;
      TRY(done(launch_head_gather(p, static_cast<int>(std::min<int64_t>(w.rows, 8 * api_sm_count())), s), "head-gather"));
    }
    if (w.copy_head) {
      HeadGatherParams p = {};
      p.N = a->V, p.D = a->D, p.pad_to = 1;
      p.in = static_cast<const uint16_t*>(a->head), p.in_stride = a->V > 1 ? a->head_stride : a->D;
      p.out = at<uint16_t>(w.head), p.out_stride = w.Dp;
      TRY(done(launch_head_gather(p, std::min(a->V, 8 * api_sm_count()), s), "head-gather"));
    }
    return SPECV_OK;
  }

  // Rows of a box of few rows (whole groups of the swizzle), or 0.
  int few_box() const { return w.half ? static_cast<int>(up_to(a->N, 8)) : 0; }
  // rows_k: the rows in use are K, not M.
  ProductParams product(int32_t M, int32_t N, int32_t K, bool rows_k) const {
    ProductParams p = {};
    p.M = M, p.N = N, p.K = K, p.batch = 1, p.splits = 1;
    p.bf16 = 1;
    p.rows = w.gather ? at<int32_t>(w.count) : nullptr;
    p.rows_k = rows_k;
    p.a_rows = rows_k ? 0 : few_box();
    return p;
  }
  specv_status head_map(CUtensorMap* m, bool mn, int64_t first, int64_t n) const {
    return operand_map(m, true, mn, head() + first * head_stride(), a->D, n, 1, head_stride(), 0);
  }

  specv_status forward() {
    ProductParams p = product(a->N, a->V, a->D, false);
    TRY(operand_map(&p.a, true, false, hidden(), a->D, a->N, 1, hidden_stride(), 0, few_box()));
    TRY(head_map(&p.b, false, 0, a->V));
    p.err = at<int32_t>(w.err);
    p.stall = api_test_stall('E');
    HeadStatsParams e = {};
    e.target = w.gather ? at<int32_t>(w.target) : a->targets;
    e.part = at<float2>(w.part), e.ld = w.ld, e.z_target = at<float>(w.z_target);
    e.V = a->V, e.c2 = a->scale * kLog2e;
    if (w.keep) {
      Out16 out = {};
      TRY(product_map(&out.map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, at<uint16_t>(w.dz), a->V, w.rows, 1, 2 * w.tokens, 0, 32));
      out.cols = a->V;
      TRY(done(launch_head_keep(p, e, out, s), "head-stats"));
    } else {
      TRY(done(launch_head_stats(p, e, s), "head-stats"));
    }
    HeadJoinParams j = {};
    j.N = a->N, j.V = a->V, j.parts = (a->V + w.part_cols - 1) / w.part_cols;
    j.part = e.part, j.z_target = e.z_target, j.ld = w.ld, j.scale = a->scale;
    j.place = w.gather ? at<int32_t>(w.place) : nullptr;
    j.target = a->targets, j.weight = a->weights, j.all = every_row();
    j.bad = w.grads ? at<int32_t>(w.bad) : nullptr;
    j.err = p.err, j.errs = w.half ? product_grid<false>(p) : product_grid<true>(p);
    j.loss = a->loss, j.stats = a->stats, j.status = a->row_status;
    j.row = w.grads ? at<HeadRow>(w.row) : nullptr, j.most = at<float>(w.most);
    return done(launch_head_join(j, s), "head-join");
  }

  specv_status backward() {
    // (TMA stores whole 16-byte words: what lies behind a row stays as it is)
    const bool tma = aligned(a->grad_head, 16) && a->grad_head_stride % 8 == 0 && a->D % 8 == 0;
    int piece = 0;
    for (int64_t v = 0; v < a->V; v += w.tokens, ++piece) {
      const int32_t n = static_cast<int32_t>(std::min<int64_t>(w.tokens, a->V - v));
      uint16_t* dz = at<uint16_t>(w.dz);
      if (w.keep) {
        HeadWeightParams p = {};
        p.N = a->N, p.V = a->V, p.count = w.gather ? at<int32_t>(w.count) : nullptr;
        p.part = at<float2>(w.part), p.ld = w.ld, p.row = at<HeadRow>(w.row), p.c2 = a->scale * kLog2e;
        p.w = dz, p.stride = w.tokens, p.part_cols = w.part_cols;
        const int64_t blocks = (w.rows * ((a->V + 255) / 256) + 7) / 8;
        TRY(done(launch_head_weight(p, static_cast<int>(std::min<int64_t>(blocks, 8 * api_sm_count())), s), "head-dz"));
      } else {  // dz of the piece
        ProductParams p = product(a->N, n, a->D, false);
        TRY(operand_map(&p.a, true, false, hidden(), a->D, a->N, 1, hidden_stride(), 0, few_box()));
        TRY(head_map(&p.b, false, v, n));
        p.late = at<int32_t>(w.late), p.stall = piece ? 0 : api_test_stall('G');
        ProbEpi::Params e = {};
        TRY(product_map(&e.out.map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dz, n, w.rows, 1, 2 * w.tokens, 0, 32));
        e.out.cols = n;
        e.row = at<HeadRow>(w.row), e.first = static_cast<int32_t>(v), e.c2 = a->scale * kLog2e;
        TRY(done(launch_head_prob(p, e, s), "head-dz"));
      }
      if (a->grad_head) {  // dW of the piece
        ProductParams p = product(n, a->D, a->N, true);
        TRY(operand_map(&p.a, true, true, dz, n, w.rows, 1, w.tokens, 0));
        TRY(operand_map(&p.b, true, true, hidden(), a->D, w.rows, 1, hidden_stride(), 0));
        p.late = at<int32_t>(w.late), p.stall = piece ? 0 : api_test_stall('H');
        Out16 e = {};
        uint16_t* out = static_cast<uint16_t*>(a->grad_head) + v * a->grad_head_stride;
        const int64_t stride = a->V > 1 ? a->grad_head_stride : up_to(a->D, 8);
        if (tma)
          TRY(product_map(&e.map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, out, a->D, n, 1, 2 * stride, 0, 32));
        else
          e.direct = out;
        e.stride = stride, e.cols = a->D;
        TRY(done(launch_head_head(p, e, at<float>(w.most), s), "head-dW"));
      }
      if (a->grad_hidden) {  // the piece's part of dh
        ProductParams p = product(a->N, a->D, n, false);
        p.splits = std::min<int>(w.splits, static_cast<int>(up_to(n, kProdBK) / kProdBK));
        TRY(operand_map(&p.a, true, false, dz, n, w.rows, 1, w.tokens, 0, few_box()));
        TRY(head_map(&p.b, true, v, n));
        p.late = at<int32_t>(w.late), p.stall = piece ? 0 : api_test_stall('I');
        SumEpi::Params e = {};
        TRY(product_map(&e.out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, at<float>(w.sum), w.Ds, w.rows, w.splits, 4 * w.Ds,
                        4 * w.rows * w.Ds, 32));
        e.cols = a->D, e.add = piece > 0, e.splits = p.splits;
        TRY(done(launch_head_hidden(p, e, s), "head-dh"));
      }
    }
    HeadFinishParams f = {};
    f.N = a->N, f.V = a->V, f.D = a->D;
    f.late = at<int32_t>(w.late), f.status = a->row_status;
    f.head = static_cast<uint16_t*>(a->grad_head), f.head_stride = a->V > 1 ? a->grad_head_stride : a->D;
    if (!a->grad_hidden) return done(launch_head_finish(f, api_sm_count(), s), "head-end");
    // (a last piece of few blocks is cut into fewer parts: its first parts are added to)
    f.splits = std::min<int>(w.splits, static_cast<int>(up_to(std::min<int64_t>(w.tokens, a->V), kProdBK) / kProdBK));
    f.sum = at<float>(w.sum), f.ld = w.Ds, f.split_stride = w.rows * w.Ds;
    f.place = w.gather ? at<int32_t>(w.place) : nullptr, f.row = at<HeadRow>(w.row), f.most = at<float>(w.most);
    f.out = static_cast<uint16_t*>(a->grad_hidden), f.stride = a->N > 1 ? a->grad_hidden_stride : a->D;
    f.vec = aligned(a->grad_hidden, 16) && f.stride % 8 == 0;
    const int64_t blocks = (static_cast<int64_t>(a->N) * ((a->D + 3) / 4) + 255) / 256;
    return done(launch_head_finish(f, static_cast<int>(std::min<int64_t>(blocks, 16 * api_sm_count())), s), "head-dh");
  }
};

// No rows: the head's gradient is an empty sum.
specv_status no_rows(const specv_head_args* a, void* stream) {
  if (a->grad_head) {
    const size_t pitch = 2 * (a->V > 1 ? a->grad_head_stride : static_cast<int64_t>(a->D));
    const cudaError_t e = cudaMemset2DAsync(a->grad_head, pitch, 0, 2 * static_cast<size_t>(a->D), a->V,
                                            static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return api_fail(SPECV_ERR_CUDA, "head-dW: %s", cudaGetErrorString(e));
  }
  return api_done(0);
}

specv_status check_space(const specv_head_args* a, const HeadSpace& w, void* workspace, size_t bytes) {
  const int64_t tiles = up_to(a->N, kProdTile) / kProdTile * ((static_cast<int64_t>(a->V) + kProdTile - 1) / kProdTile);
  const int64_t wide = (static_cast<int64_t>(a->V) + kProdTile - 1) / kProdTile * (up_to(a->D, kProdTile) / kProdTile);
  if (std::max(tiles, wide) > (1 << 30)) return api_fail(SPECV_ERR_UNSUPPORTED, "N, V and D too large");
  if (!workspace || bytes < w.bytes)
    return api_fail(SPECV_ERR_WORKSPACE, "workspace of %zu bytes needed, got %zu", w.bytes, workspace ? bytes : 0);
  if (!aligned(workspace, 256)) return api_fail(SPECV_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
  return SPECV_OK;
}

}  // namespace

extern "C" {

size_t specv_head_workspace_bytes(const specv_head_args* a) {
  if (!a || a->N < 1 || a->V < 1 || a->D < 1) return 0;
  return std::max(head_space(a, true).bytes, head_space(a, false).bytes);
}

specv_status specv_head_loss(const specv_head_args* a, void* workspace, size_t workspace_bytes, void* stream) {
  api_done(0);
  TRY(check_head(a));
  if (a->grad_loss) return api_fail(SPECV_ERR_INVALID_ARG, "grad_loss belongs to specv_head_loss_backward");
  if (a->N == 0) return no_rows(a, stream);
  if (!a->loss) return api_fail(SPECV_ERR_INVALID_ARG, "a required pointer is NULL");
  HeadRun run = {a, head_space(a, true), static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream)};
  TRY(check_space(a, run.w, workspace, workspace_bytes));
  TRY(run.rows(false));
  TRY(run.forward());
  if (run.w.grads) TRY(run.backward());
  return api_done(run.launches);
}

specv_status specv_head_loss_backward(const specv_head_args* a, void* workspace, size_t workspace_bytes, void* stream) {
  api_done(0);
  TRY(check_head(a));
  if (a->N == 0) return no_rows(a, stream);
  if (!a->stats || (!a->grad_hidden && !a->grad_head)) return api_fail(SPECV_ERR_INVALID_ARG, "a required pointer is NULL");
  HeadRun run = {a, head_space(a, false), static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream)};
  TRY(check_space(a, run.w, workspace, workspace_bytes));
  TRY(run.rows(true));
  TRY(run.backward());
  return api_done(run.launches);
}

}  // extern "C"
