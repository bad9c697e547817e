/* zslayer.h -- C ABI of libzshard, third part: the layers whose parameters'
 * gradients are sums over a rank's tokens.  A norm's weights and an embedding
 * table take no matrix product: their forward passes read the working copy that
 * the step writes, and their backward passes write, or add to, the gradients
 * that the step reads (zs_adamw_piece.grads, zs_shard_args.grads), at any
 * alignment and in any of their types.
 *
 * zshard.h's conventions hold for every call here: device memory is the
 * caller's, nothing is allocated, argument structs are host memory read during
 * the call, calls are asynchronous on `stream` (a stream of the current
 * device) and can be captured, argument errors are returned before anything is
 * launched.  Calls on different streams may not share a workspace; a workspace
 * needs no initialisation and holds nothing between calls.
 *
 * Numerics.  Every element is widened to fp32 and each output rounded once, to
 * nearest even.  The fp32 operations are those written below, each rounded
 * once (correctly rounded division and root); only a product that goes straight
 * into a sum over a row or over rows is not rounded before it is added.  Such
 * sums are in an order that is fixed by the call's sizes and types, whether it
 * is in place, and the device: the same bits every time.  Infinities and NaN
 * propagate by IEEE rules, within their row and into the gradients' sums.
 *
 * Rows of activations are row-major with a stride in elements, at least cols;
 * what lies between two rows is neither read nor written.  Element types are
 * ZS_F16, ZS_BF16 or ZS_F32 each; an address is a multiple of its element's
 * size, and accesses are fastest where rows begin on 16 bytes. */
#ifndef ZSLAYER_H
#define ZSLAYER_H

#include "zsadamw.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ZS_NORM_MAX_COLS 16384

typedef enum { ZS_NORM_LAYER = 0, ZS_NORM_RMS = 1 } zs_norm_kind;
typedef enum { ZS_I32 = 4, ZS_I64 = 5 } zs_id_dtype;

/* Layer norm (Ba, Kiros & Hinton, "Layer Normalization", 2016) or root-mean-
 * square norm (Zhang & Sennrich, "Root Mean Square Layer Normalization",
 * 2019) of each row, after the residual addition if there is one:
 *   t = x, or RN(x + residual), which goes to `total`
 *   layer: mu = sum(t) / cols, var = sum((t - mu)^2) / cols
 *   rms:   mu = 0,             var = sum(t^2) / cols
 *   rstd = 1 / sqrt(var + eps)
 *   y = RN(((t - mu) * rstd) * gamma + beta)
 * The norm is of t as it is stored, so that the backward pass can start from
 * `total`. */
typedef struct {
  int64_t rows;            /* >= 0 */
  int64_t cols;            /* 1..ZS_NORM_MAX_COLS */
  int32_t kind;            /* zs_norm_kind */
  int32_t dtype;           /* of x, residual, total and y */
  int32_t w_dtype;         /* of gamma and beta */
  int32_t reserved;        /* 0 */
  double eps;              /* >= 0; used as fp32, finite there */
  const void* x;
  const void* residual;    /* or NULL: t = x, and total is not looked at */
  void* total;             /* written where there is a residual */
  void* y;                 /* written */
  int64_t x_stride, residual_stride, total_stride, y_stride;
  const void* gamma;       /* cols, or NULL: ones */
  const void* beta;        /* cols, or NULL: zeros */
  float* mean;             /* rows, written, or NULL; not looked at for ZS_NORM_RMS */
  float* rstd;             /* rows, written, or NULL */
  void* stream;
} zs_norm_args;

/* Bytes per element: 2 (4 with a residual) elements of dtype.  In place: total
 * or y may be x or residual itself (same address and stride; not both the
 * same).  Errors: ZS_ERR_NULL, ZS_ERR_ARG (rows, cols < 1, kind, eps, a
 * stride, a misaligned address, reserved), ZS_ERR_DTYPE, ZS_ERR_RANGE (cols
 * above ZS_NORM_MAX_COLS, or more memory than addresses reach), ZS_ERR_ALIAS
 * (an output meets another output or, but for in place, an input),
 * ZS_ERR_HIP. */
zs_status zs_norm_forward(const zs_norm_args* args);

/* The gradients of that norm, for dy at y:
 *   h = (x - mean) * rstd (rms: x * rstd),  a = dy * gamma
 *   c1 = sum(a) / cols (rms: 0),  c2 = sum(a * h) / cols
 *   dx = RN(((a - c1) - h * c2) * rstd + dres)
 *   dgamma = RN((accumulate: dgamma +) sum over rows of dy * h)
 *   dbeta  = RN((accumulate: dbeta +) sum over rows of dy)
 * x is what was normalised (the forward pass's total where it had a residual),
 * mean and rstd are the forward pass's.  dres: the gradient that reaches the
 * same sum past the norm, so that dx is that of both x and the residual. */
typedef struct {
  int64_t rows, cols;
  int32_t kind;
  int32_t dtype;           /* of dy, x, dres and dx */
  int32_t w_dtype;         /* of gamma */
  int32_t grad_dtype;      /* of dgamma and dbeta */
  int32_t accumulate;      /* 1: dgamma and dbeta are added to; 0: written */
  int32_t reserved;        /* 0 */
  const void* dy;
  const void* x;
  const void* dres;        /* or NULL */
  void* dx;                /* written */
  int64_t dy_stride, x_stride, dres_stride, dx_stride;
  const void* gamma;       /* or NULL: ones */
  const float* mean;       /* not looked at for ZS_NORM_RMS */
  const float* rstd;
  void* dgamma;            /* cols, or NULL: not wanted */
  void* dbeta;             /* cols, or NULL: not wanted */
  void* workspace;         /* only if dgamma or dbeta is wanted */
  size_t workspace_bytes;
  void* stream;
} zs_norm_grad_args;

/* Device bytes for the sums of zs_norm_backward's gradients: 4 KiB for each of
 * cols rounded up to a power of two, 512 at least, whatever the rows; 0 on sizes
 * that it refuses. */
size_t zs_norm_workspace_bytes(int64_t rows, int64_t cols);

/* Bytes per element: 3 (4 with dres) elements of dtype.  In place: dx may be
 * dy, x or dres itself.  No rows: dgamma and dbeta are still written.
 * Errors: as zs_norm_forward, and ZS_ERR_CAPACITY (the workspace is too small
 * or not 256-byte aligned). */
zs_status zs_norm_backward(const zs_norm_grad_args* args);

/* The lookup of tokens' rows in an embedding table, scaled, and a second
 * lookup added to it (positions):
 *   y[t] = RN(f32(scale) * table[ids[t] - first_row] + pos_table[pos_ids[t]])
 * An id without a row in the table (below first_row, or first_row + rows or
 * above: padding, or another rank's part of a vocabulary that is cut over
 * ranks) gives +0 in the place of the product, and a position outside
 * [0, pos_rows) nothing to add.  Without pos_table the product alone is
 * rounded. */
typedef struct {
  int64_t tokens;          /* >= 0 */
  int64_t rows, cols;      /* of the table; >= 1 */
  int64_t first_row;       /* the id of the table's first row, >= 0 */
  int32_t id_dtype;        /* zs_id_dtype, of ids and pos_ids */
  int32_t dtype;           /* of y */
  int32_t table_dtype;     /* of table and pos_table */
  int32_t reserved;        /* 0 */
  double scale;            /* used as fp32, finite there */
  const void* ids;
  const void* table;       /* rows x cols, contiguous */
  void* y;                 /* tokens rows, written */
  int64_t y_stride;
  const void* pos_ids;     /* with pos_table */
  const void* pos_table;   /* pos_rows x cols, contiguous, or NULL */
  int64_t pos_rows;
  void* stream;
} zs_embed_args;

#define ZS_EMBED_MAX_TOKENS (1 << 28)
#define ZS_EMBED_MAX_ROWS ((int64_t)1 << 30)
#define ZS_EMBED_MAX_COLS (1 << 20)

/* Errors: ZS_ERR_NULL, ZS_ERR_ARG, ZS_ERR_DTYPE, ZS_ERR_RANGE (more tokens,
 * rows or columns than the limits above), ZS_ERR_ALIAS (y meets an input),
 * ZS_ERR_HIP. */
zs_status zs_embed_forward(const zs_embed_args* args);

/* The table's gradient for dy at y:
 *   grad[r] = RN((accumulate: grad[r] +) f32(scale) * sum over t with
 *             ids[t] - first_row = r, in the order of t, of dy[t])
 * accumulate 0 writes all rows, zeros where no token names one; 1 reads and
 * writes only the rows that a token names (a table tied to the output
 * projection, micro batches).  Ids without a row add nothing, and their dy is
 * not read.  The gradient of a position table is this call with pos_ids. */
typedef struct {
  int64_t tokens;
  int64_t rows, cols;
  int64_t first_row;
  int32_t id_dtype;
  int32_t dtype;           /* of dy */
  int32_t grad_dtype;      /* of grad */
  int32_t accumulate;
  double scale;            /* used as fp32, finite there */
  const void* ids;
  const void* dy;          /* tokens rows */
  int64_t dy_stride;
  void* grad;              /* rows x cols, contiguous; written or added to */
  void* workspace;
  size_t workspace_bytes;
  void* stream;
} zs_embed_grad_args;

/* Device bytes for zs_embed_backward (the tokens in the order of their rows,
 * and the sums of rows whose tokens are summed in several parts), of so many
 * tokens or fewer and of so many columns: a buffer for the longest batch does
 * for all.  0 on sizes that it refuses. */
size_t zs_embed_workspace_bytes(int64_t tokens, int64_t rows, int64_t cols);

/* Errors: as zs_embed_forward, and ZS_ERR_CAPACITY (the workspace is smaller
 * than what this many tokens take, or not 256-byte aligned). */
zs_status zs_embed_backward(const zs_embed_grad_args* args);

#ifdef __cplusplus
}
#endif

#endif /* ZSLAYER_H */
