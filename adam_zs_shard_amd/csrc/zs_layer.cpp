// zs_layer.cpp -- host side of the layer operators: argument checks and
// workspace sizes.  Every argument error is returned before anything touches
// the device.

#include <hip/hip_runtime_api.h>

#include <cmath>

#include "zs_layer.h"

namespace {

using zs::Rows;
using zs::kNormParts;

constexpr int64_t kMaxBytes = int64_t{1} << 56;

bool dtype_ok(int32_t dt) { return dt == ZS_F16 || dt == ZS_BF16 || dt == ZS_F32; }
int64_t size_of(int32_t dt) { return dt == ZS_F32 ? 4 : 2; }
// Whether the fp32 value that the kernels use is finite.
bool f32_finite(double x) { return std::isfinite(static_cast<float>(x)); }

zs_status from_hip(hipError_t e) {
  return e == hipSuccess ? ZS_OK : static_cast<zs_status>(zs::hip_status(e));
}

// Memory that a call reads or writes: `width` bytes of each row, `pitch` apart.
struct Span {
  uintptr_t lo, hi;
  int64_t width, pitch;
  bool written;
};

bool meet(const Span& a, const Span& b) {
  if (a.hi <= b.lo || b.hi <= a.lo) return false;
  if (a.pitch != b.pitch) return true;
  // columns of one wider buffer: apart in the first row, apart in all
  const uintptr_t pitch = static_cast<uintptr_t>(a.pitch);
  const uintptr_t d = b.lo >= a.lo ? (b.lo - a.lo) % pitch
                                   : (pitch - (a.lo - b.lo) % pitch) % pitch;
  return d < static_cast<uintptr_t>(a.width) || d + static_cast<uintptr_t>(b.width) > pitch;
}

// The operands of a call, checked one by one; the first error stays.
class Operands {
 public:
  // `count` elements, or `rows` rows of `cols` elements; optional operands are
  // not given at all.
  void vector(const void* at, int64_t count, int64_t size, bool written) {
    rows(at, 1, count, count, size, written, nullptr);
  }
  void rows(const void* at, int64_t n, int64_t cols, int64_t stride, int64_t size, bool written,
            Rows* out) {
    if (status_ != ZS_OK || n == 0) return;
    if (!at) return fail(ZS_ERR_NULL);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(at);
    if (stride < cols || lo % static_cast<uintptr_t>(size) != 0) return fail(ZS_ERR_ARG);
    if (cols > kMaxBytes / size || (n > 1 && stride > kMaxBytes / size / (n - 1)))
      return fail(ZS_ERR_RANGE);
    const int64_t bytes = ((n - 1) * stride + cols) * size;
    if (lo > UINTPTR_MAX - static_cast<uintptr_t>(bytes)) return fail(ZS_ERR_RANGE);
    // one row has no stride: one that all rows share is made up
    spans_[count_++] = {lo, lo + static_cast<uintptr_t>(bytes), cols * size,
                        n > 1 ? stride * size : 0, written};
    if (out) *out = {lo, stride * size};
  }
  zs_status status() const { return status_; }
  // Whether what is written keeps clear of everything else; `in_place`: an
  // output may be an input itself.
  zs_status apart(bool in_place) {
    if (status_ != ZS_OK) return status_;
    for (int i = 0; i < count_; ++i)
      for (int j = 0; j < count_; ++j) {
        const Span &w = spans_[i], &s = spans_[j];
        if (i == j || !w.written) continue;
        const bool same = w.lo == s.lo && w.hi == s.hi && w.pitch == s.pitch && w.width == s.width;
        if (in_place && same && !s.written && i < rows_ && j < rows_) continue;
        if (clash(w, s)) return ZS_ERR_ALIAS;
      }
    return ZS_OK;
  }
  // The operands given so far are rows of activations, which outputs among them
  // may share with inputs among them.
  void end_of_rows() { rows_ = count_; }

 private:
  void fail(zs_status s) { status_ = s; }
  static bool clash(const Span& a, const Span& b) {
    if (a.pitch == 0 || b.pitch == 0) return a.lo < b.hi && b.lo < a.hi;
    return meet(a, b);
  }
  Span spans_[16];
  int count_ = 0, rows_ = 0;
  zs_status status_ = ZS_OK;
};

zs_status norm_sizes(int64_t rows, int64_t cols, int32_t kind) {
  if (rows < 0 || cols < 1 || (kind != ZS_NORM_LAYER && kind != ZS_NORM_RMS)) return ZS_ERR_ARG;
  if (cols > ZS_NORM_MAX_COLS || rows > kMaxBytes) return ZS_ERR_RANGE;
  return ZS_OK;
}

size_t norm_workspace(int64_t cols) {
  return sizeof(float) * 2 * kNormParts * static_cast<size_t>(zs::norm_width(static_cast<int>(cols)));
}

zs_status workspace_ok(const void* at, size_t bytes, size_t need) {
  if (!at) return ZS_ERR_NULL;
  return reinterpret_cast<uintptr_t>(at) % 256u != 0 || bytes < need ? ZS_ERR_CAPACITY : ZS_OK;
}

zs_status norm_forward(const zs_norm_args* q) {
  if (!q) return ZS_ERR_NULL;
  if (const zs_status st = norm_sizes(q->rows, q->cols, q->kind)) return st;
  if (!f32_finite(q->eps) || q->eps < 0.0 || q->reserved != 0) return ZS_ERR_ARG;
  if (!dtype_ok(q->dtype) || !dtype_ok(q->w_dtype)) return ZS_ERR_DTYPE;
  if (q->rows == 0) return ZS_OK;
  const int64_t size = size_of(q->dtype), wsize = size_of(q->w_dtype);
  const bool layer = q->kind == ZS_NORM_LAYER;
  zs::NormLaunch L{};
  Operands o;
  o.rows(q->x, q->rows, q->cols, q->x_stride, size, false, &L.x);
  if (q->residual) {
    o.rows(q->residual, q->rows, q->cols, q->residual_stride, size, false, &L.residual);
    o.rows(q->total, q->rows, q->cols, q->total_stride, size, true, &L.total);
  }
  o.rows(q->y, q->rows, q->cols, q->y_stride, size, true, &L.y);
  o.end_of_rows();
  if (q->gamma) o.vector(q->gamma, q->cols, wsize, false);
  if (q->beta) o.vector(q->beta, q->cols, wsize, false);
  if (layer && q->mean) o.vector(q->mean, q->rows, 4, true);
  if (q->rstd) o.vector(q->rstd, q->rows, 4, true);
  if (const zs_status st = o.apart(true)) return st;
  L.rows = q->rows;
  L.cols = static_cast<int>(q->cols);
  L.dt = q->dtype;
  L.wdt = q->w_dtype;
  L.layer = layer;
  L.eps = static_cast<float>(q->eps);
  L.gamma = q->gamma;
  L.beta = q->beta;
  L.mean = layer ? q->mean : nullptr;
  L.rstd = q->rstd;
  L.stream = static_cast<hipStream_t>(q->stream);
  return from_hip(zs::launch_norm(L));
}

zs_status norm_backward(const zs_norm_grad_args* q) {
  if (!q) return ZS_ERR_NULL;
  if (const zs_status st = norm_sizes(q->rows, q->cols, q->kind)) return st;
  if ((q->accumulate != 0 && q->accumulate != 1) || q->reserved != 0) return ZS_ERR_ARG;
  if (!dtype_ok(q->dtype) || !dtype_ok(q->w_dtype) || !dtype_ok(q->grad_dtype)) return ZS_ERR_DTYPE;
  if (q->rows == 0 && (q->accumulate || (!q->dgamma && !q->dbeta))) return ZS_OK;
  const int64_t size = size_of(q->dtype), gsize = size_of(q->grad_dtype);
  const bool layer = q->kind == ZS_NORM_LAYER;
  zs::NormGradLaunch L{};
  Operands o;
  o.rows(q->dy, q->rows, q->cols, q->dy_stride, size, false, &L.dy);
  o.rows(q->x, q->rows, q->cols, q->x_stride, size, false, &L.x);
  if (q->dres) o.rows(q->dres, q->rows, q->cols, q->dres_stride, size, false, &L.dres);
  o.rows(q->dx, q->rows, q->cols, q->dx_stride, size, true, &L.dx);
  o.end_of_rows();
  if (q->gamma) o.vector(q->gamma, q->cols, size_of(q->w_dtype), false);
  if (q->rows > 0) {
    if (layer) o.vector(q->mean, q->rows, 4, false);
    o.vector(q->rstd, q->rows, 4, false);
  }
  if (q->dgamma) o.vector(q->dgamma, q->cols, gsize, true);
  if (q->dbeta) o.vector(q->dbeta, q->cols, gsize, true);
  if (q->dgamma || q->dbeta) {
    if (o.status() == ZS_OK)
      if (const zs_status st = workspace_ok(q->workspace, q->workspace_bytes, norm_workspace(q->cols)))
        return st;
    o.vector(q->workspace, static_cast<int64_t>(norm_workspace(q->cols)), 1, true);
  }
  if (const zs_status st = o.apart(true)) return st;
  L.rows = q->rows;
  L.cols = static_cast<int>(q->cols);
  L.dt = q->dtype;
  L.wdt = q->w_dtype;
  L.gdt = q->grad_dtype;
  L.layer = layer;
  L.accumulate = q->accumulate != 0;
  L.gamma = q->gamma;
  L.mean = layer ? q->mean : nullptr;
  L.rstd = q->rstd;
  L.dgamma = q->dgamma;
  L.dbeta = q->dbeta;
  L.partial = static_cast<float*>(q->workspace);
  L.stream = static_cast<hipStream_t>(q->stream);
  return from_hip(zs::launch_norm_grad(L));
}

zs_status embed_sizes(int64_t tokens, int64_t rows, int64_t cols) {
  if (tokens < 0 || rows < 1 || cols < 1) return ZS_ERR_ARG;
  if (tokens > ZS_EMBED_MAX_TOKENS || rows > ZS_EMBED_MAX_ROWS || cols > ZS_EMBED_MAX_COLS)
    return ZS_ERR_RANGE;
  return ZS_OK;
}

bool id_dtype_ok(int32_t dt) { return dt == ZS_I32 || dt == ZS_I64; }

zs_status embed_forward(const zs_embed_args* q) {
  if (!q) return ZS_ERR_NULL;
  if (const zs_status st = embed_sizes(q->tokens, q->rows, q->cols)) return st;
  if (q->first_row < 0 || !f32_finite(q->scale) || q->reserved != 0) return ZS_ERR_ARG;
  if (q->pos_table && q->pos_rows < 1) return ZS_ERR_ARG;
  if (q->pos_table && q->pos_rows > ZS_EMBED_MAX_ROWS) return ZS_ERR_RANGE;
  if (!dtype_ok(q->dtype) || !dtype_ok(q->table_dtype) || !id_dtype_ok(q->id_dtype)) return ZS_ERR_DTYPE;
  if (q->tokens == 0) return ZS_OK;
  const int64_t isize = q->id_dtype == ZS_I64 ? 8 : 4, tsize = size_of(q->table_dtype);
  zs::EmbedLaunch L{};
  Operands o;
  o.rows(q->y, q->tokens, q->cols, q->y_stride, size_of(q->dtype), true, &L.y);
  o.vector(q->ids, q->tokens, isize, false);
  o.vector(q->table, q->rows * q->cols, tsize, false);
  if (q->pos_table) {
    o.vector(q->pos_ids, q->tokens, isize, false);
    o.vector(q->pos_table, q->pos_rows * q->cols, tsize, false);
  }
  if (const zs_status st = o.apart(false)) return st;
  L.tokens = q->tokens;
  L.rows = q->rows;
  L.first_row = q->first_row;
  L.pos_rows = q->pos_rows;
  L.cols = static_cast<int>(q->cols);
  L.dt = q->dtype;
  L.tdt = q->table_dtype;
  L.wide_ids = q->id_dtype == ZS_I64;
  L.scale = static_cast<float>(q->scale);
  L.ids = q->ids;
  L.table = q->table;
  L.pos_ids = q->pos_ids;
  L.pos_table = q->pos_table;
  L.stream = static_cast<hipStream_t>(q->stream);
  return from_hip(zs::launch_embed(L));
}

zs_status embed_backward(const zs_embed_grad_args* q) {
  if (!q) return ZS_ERR_NULL;
  if (const zs_status st = embed_sizes(q->tokens, q->rows, q->cols)) return st;
  if (q->first_row < 0 || !f32_finite(q->scale) || (q->accumulate != 0 && q->accumulate != 1))
    return ZS_ERR_ARG;
  if (!dtype_ok(q->dtype) || !dtype_ok(q->grad_dtype) || !id_dtype_ok(q->id_dtype)) return ZS_ERR_DTYPE;
  if (q->tokens == 0 && q->accumulate) return ZS_OK;
  zs::EmbedGradLaunch L{};
  Operands o;
  o.rows(q->dy, q->tokens, q->cols, q->dy_stride, size_of(q->dtype), false, &L.dy);
  if (q->tokens > 0) o.vector(q->ids, q->tokens, q->id_dtype == ZS_I64 ? 8 : 4, false);
  o.vector(q->grad, q->rows * q->cols, size_of(q->grad_dtype), true);
  if (q->tokens > 0) {
    const size_t need = zs::embed_layout(q->tokens, q->cols).total;
    if (o.status() == ZS_OK)
      if (const zs_status st = workspace_ok(q->workspace, q->workspace_bytes, need)) return st;
    o.vector(q->workspace, static_cast<int64_t>(need), 1, true);
  }
  if (const zs_status st = o.apart(false)) return st;
  L.tokens = q->tokens;
  L.rows = q->rows;
  L.first_row = q->first_row;
  L.cols = static_cast<int>(q->cols);
  L.dt = q->dtype;
  L.gdt = q->grad_dtype;
  L.wide_ids = q->id_dtype == ZS_I64;
  L.accumulate = q->accumulate != 0;
  L.scale = static_cast<float>(q->scale);
  L.ids = q->ids;
  L.grad = q->grad;
  L.workspace = static_cast<unsigned char*>(q->workspace);
  L.stream = static_cast<hipStream_t>(q->stream);
  return from_hip(zs::launch_embed_grad(L));
}

}  // namespace

extern "C" {

zs_status zs_norm_forward(const zs_norm_args* args) {
  return zs::guard([&] { return norm_forward(args); });
}

size_t zs_norm_workspace_bytes(int64_t rows, int64_t cols) {
  return norm_sizes(rows, cols, ZS_NORM_LAYER) == ZS_OK ? norm_workspace(cols) : 0;
}

zs_status zs_norm_backward(const zs_norm_grad_args* args) {
  return zs::guard([&] { return norm_backward(args); });
}

zs_status zs_embed_forward(const zs_embed_args* args) {
  return zs::guard([&] { return embed_forward(args); });
}

size_t zs_embed_workspace_bytes(int64_t tokens, int64_t rows, int64_t cols) {
  if (embed_sizes(tokens, rows, cols) != ZS_OK) return 0;
  return zs::embed_workspace(tokens > 0 ? tokens : 1, cols);
}

zs_status zs_embed_backward(const zs_embed_grad_args* args) {
  return zs::guard([&] { return embed_backward(args); });
}

}  // extern "C"
