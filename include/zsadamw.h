/* zsadamw.h -- C ABI of libzshard, second part: AdamW over many tensors, with
 * the moments in 32 or in 8 bits, clipping by the global norm, and what a
 * training loop needs around it.
 *
 * zshard.h's conventions hold for every call here: device memory is the
 * caller's, nothing is allocated, descriptor structs are host memory read
 * during the call, calls are asynchronous on `stream` (a stream of the current
 * device), argument errors are returned before anything is launched, and the
 * fp32 arithmetic is the stated sequence with every operation rounded once.
 *
 * What one step computes for each element of each tensor (decoupled weight
 * decay: Loshchilov & Hutter, "Decoupled Weight Decay Regularization", 2019):
 *   g  = ((sum over ranks r = 0..p-1, in that order, of grad_r) / p) * gs
 *   m' = beta1*m + (1-beta1)*g,   v' = beta2*v + (1-beta2)*g*g
 *   u  = m_hat / (sqrt(v_hat) + eps)
 *   w' = w - (lr_i*u + (lr_i*decay_i)*w),   lr_i = lr * the tensor's lr_scale
 *   param = w' rounded to nearest-even fp16/bf16
 * With 32-bit states m_hat = m'/(1-beta1^t) and v_hat = v'/(1-beta2^t): with
 * no decay, no clipping and lr_scale 1 the step is ZS_ADAM_STANDARD's, bit
 * for bit.  With 8-bit states lr_i*u is f32(lr_i/(1-beta1^t)) * (m' /
 * (sqrt(v') * f32(1/sqrt(1-beta2^t)) + eps)), from the moments before they
 * are rounded, where the root and the reciprocal are the hardware's, within
 * 1 ulp each, and a v' or a divisor below 2^-126 may count as 0.
 * gs = f32(grad_scale * coef), coef = min(1, max_norm / (sqrt(sumsq) *
 * |grad_scale| + 1e-6)) in double where a norm is given, else 1.
 *
 * Moments in 8 bits.  A tensor's moments are cut into blocks of
 * ZS_STATE8_BLOCK elements from its first one; each block has one fp32 scale
 * per moment, and a value is its code times the scale.  m: OCP e4m3 codes,
 * scale = max|m'| * f32(1/448).  v: OCP e5m2 codes, scale = max v' *
 * f32(1/57344).  Codes are those of x * f32(top / max) cut to [-top, top]:
 * m is off by at most 1/16 and sqrt(v) by about as much (twice that with
 * random rounding), whatever a value's size within 2^14 (m) or 2^29 (v) of its
 * block's largest.  A positive v
 * never gets code 0, since the update divides by its root.  A block whose
 * largest value is below 2^-110 is held as zeros; one that holds an infinity
 * or NaN gets a NaN scale and codes 0, so that all of it reads as NaN (see
 * skip_nonfinite).  All codes and scales zero is the zero state.
 *   ZS_ROUND_NEAREST: ties to even.  The bounds above are those of one
 *     rounding.  Over a run, a step that changes a moment by less than half its
 *     codes' spacing (1/16 to 1/8 of v, 1/32 to 1/16 of m) leaves the code as
 *     it is, for good: v stops where (1-beta2)*|g*g - v| is below that, and at
 *     a beta2 of 0.95 or more a v whose gradient is gone never decays but with
 *     its block's scale.  With a constant gradient in a block whose scale
 *     another element holds, v began at 0.4 g*g and stayed at 0.42 g*g, at
 *     beta2 = 0.95, 0.99 and 0.999 alike; with Gaussian gradients from the zero
 *     state the mean root of v stood 4% (0.95, 600 steps), 30% (0.99, 1000)
 *     and 7% (0.999, 3000) too high, where random rounding stayed within 2%.
 *     It is for conversions and for comparing; training takes the other.
 *   ZS_ROUND_STOCHASTIC: up or down with the probability that the place
 *     between the two neighbours says, so that the mean of what is stored is
 *     the value itself, and small steps add up.  (Not of a positive v below
 *     the smallest code, 2^-16 / 57344 of its block's largest: it is held as
 *     that code, since code 0 is not for it.)  The random bits come from
 *     Philox4x32-7 (Salmon et al., "Parallel random numbers: as easy as 1, 2,
 *     3", SC'11) with key = seed and counter = (index of the first of four
 *     elements, step), the fours counted from the piece's first element; word
 *     j goes to element j of the four, its low 16 bits r to m, its high 16 to
 *     v.  So pieces that are cut out of a tensor at multiples of 4, with
 *     indexes to match, get the bits of the whole, and at multiples of
 *     ZS_STATE8_BLOCK its blocks, codes and scales too; cut elsewhere, their
 *     bits are others, as good.  |y| (moved up by 2^-6 for m, 2^-14 for v,
 *     where it lies below that: the even part of the grid) has
 *     r * 2^(d-16) + 2^(d-17) added to its fp32 bits and the low d bits cut,
 *     d = 20 for m, 21 for v.
 */
#ifndef ZSADAMW_H
#define ZSADAMW_H

#include "zshard.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ZS_F32 3             /* a gradient dtype of these calls: e.g. a stored fp32 mean */
#define ZS_STATE8_BLOCK 256

typedef enum { ZS_ROUND_NEAREST = 0, ZS_ROUND_STOCHASTIC = 1 } zs_rounding;
typedef enum { ZS_STATE8_M = 0, ZS_STATE8_V = 1 } zs_state8_kind;

/* One tensor (or a shard's piece of one).  Every address is that of the
 * tensor's first element, a multiple of its element size. */
typedef struct {
  int64_t len;              /* elements, >= 1 */
  float* w;                 /* fp32 master weights, updated */
  void* m;                  /* fp32 or e4m3 codes, updated */
  void* v;                  /* fp32 or e5m2 codes, updated */
  float* m_scale;           /* 8-bit states: ceil(len / ZS_STATE8_BLOCK) scales each, updated */
  float* v_scale;
  void* param;              /* 16-bit working copy, written */
  float* g_mean;            /* fp32 gradient mean, written by zs_grad_sumsq_multi if asked; else NULL */
  const void* const* grads; /* host array of p device pointers, rank order */
  double weight_decay;      /* finite, >= 0 */
  double lr_scale;          /* finite */
  int64_t index;            /* >= 0: index of element 0 for ZS_ROUND_STOCHASTIC, e.g. in the whole model
                             * (pieces of equal index share their random bits) */
} zs_adamw_piece;

/* Host-side handle of an uploaded table. */
typedef struct {
  void* workspace;
  int64_t nchunks;
  int64_t chunk_elems;
  int32_t npieces;
  int32_t p;
  int32_t grad_dtype;   /* zs_dtype or ZS_F32 */
  int32_t param_dtype;  /* zs_dtype, or 0: no working copy */
  int32_t state_bits;   /* 32, 8, or 0: gradients only */
  int32_t has_mean;     /* every piece has g_mean */
  int32_t on_lines;     /* every w, m, v and param begins on a 128-byte line */
  int32_t reserved;
} zs_adamw_table;

/* Device bytes that zs_adamw_upload needs for tensors of lens[0..npieces)
 * elements and p ranks; 0 on bad arguments. */
size_t zs_adamw_workspace_bytes(const int64_t* lens, int32_t npieces, int32_t p);

/* Writes the launch table of the tensors into the caller's device workspace
 * (256-byte aligned) with one copy on `stream`, and waits for it (call it
 * before capture).  Call once per plan: the table stays valid while the memory
 * that it names does.  One table may be used by one stream at a time
 * (zs_grad_sumsq_multi keeps its partial sums in the workspace).
 * Tensors may begin anywhere; steps are fastest where the arrays of a tensor
 * all begin on a 128-byte line or the same number of elements past one.  With
 * 8-bit states only the caller can see to that (blocks are counted from the
 * tensor's first element): 10% on 1.0e9 elements.
 *  state_bits: 32 or 8; 0 for a table of gradients only (zs_grad_sumsq_multi),
 *     whose w, m, v, param and scales are not looked at.
 *  param_dtype: ZS_F16 or ZS_BF16; 0 for no working copy.
 * Errors: ZS_ERR_NULL, ZS_ERR_ARG (p outside 1..ZS_MAX_P, state_bits, a len,
 * index, weight_decay or lr_scale out of range, an address that is no multiple
 * of its element size), ZS_ERR_RANGE (more than one launch holds: about 1.7e10
 * elements or, in short tensors, 1.6e7 of them), ZS_ERR_DTYPE, ZS_ERR_CAPACITY
 * (the workspace is too small or misaligned), ZS_ERR_ALIAS (what one tensor has
 * written overlaps what any tensor has written or read, or the workspace),
 * ZS_ERR_HIP, ZS_ERR_RESOURCE. */
zs_status zs_adamw_upload(const zs_adamw_piece* pieces, int32_t npieces, int32_t p,
                          int32_t grad_dtype, int32_t param_dtype, int32_t state_bits,
                          void* workspace, size_t ws_bytes, void* stream, zs_adamw_table* table);

typedef struct {
  double lr;          /* finite */
  double beta1;       /* in [0, 1) */
  double beta2;       /* in [0, 1) */
  double eps;         /* finite, >= 0 */
  int64_t step;       /* t >= 1: the 1-based step being produced */
  double grad_scale;  /* finite, not 0: e.g. 1 / the loss scale */
  double max_norm;    /* > 0: clip to this global norm (needs sumsq); 0: no clipping */
  uint64_t seed;      /* ZS_ROUND_STOCHASTIC */
  int32_t rounding;   /* zs_rounding, 8-bit states only */
  int32_t skip_nonfinite; /* 1: a sumsq that is infinite or NaN leaves everything as it is (needs sumsq) */
} zs_adamw_hparams;

/* The constants of a run of steps in device memory, for launches that are
 * captured once and replayed (compare zs_step_table): entry i holds step
 * first_step + i, whose learning rate may follow a schedule. */
typedef struct {
  void* dev;
  int64_t first_step;
  int32_t nsteps;
  int32_t reserved; /* 0 */
} zs_adamw_steps;

/* One AdamW step over every tensor of the table, in one launch.  sumsq: a
 * device double, the sum of squares of the whole model's mean gradient before
 * grad_scale (zs_grad_sumsq_multi, summed over the shards), or NULL.
 * Bytes per element: p gradients + 4 + 4 (w) + 2 (param) + 16 (32-bit
 * states) or 4.0625 (8-bit).  Elements beyond a tensor's len are not touched.
 * A table of no tensors returns ZS_OK without launching.
 * Errors: ZS_ERR_NULL, ZS_ERR_ARG, ZS_ERR_DTYPE, ZS_ERR_HIP. */
zs_status zs_adamw_step_multi(const zs_adamw_table* table, const zs_adamw_hparams* hp,
                              const double* sumsq, void* stream);

/* zs_adamw_step_multi with lr, beta1, beta2, eps and step from the step table's
 * current entry, read on the device (hp's own are still checked; the rest of
 * hp holds as there).  Captured as [zs_grad_sumsq_multi, this,
 * zs_adamw_steps_advance], a graph replays consecutive steps.  Past the
 * table's end nothing is updated and its `exhausted` is set. */
zs_status zs_adamw_step_multi_dev(const zs_adamw_table* table, const zs_adamw_steps* steps,
                                  const zs_adamw_hparams* hp, const double* sumsq, void* stream);

/* Device bytes of a step table of nsteps entries (0 if nsteps is outside
 * 1..ZS_MAX_TABLE_STEPS). */
size_t zs_adamw_steps_bytes(int32_t nsteps);

/* Fills a step table for steps hp->step .. hp->step + nsteps - 1 with hp's
 * betas and eps and, per step, lrs[i] (a host array) or, if lrs is NULL, hp's
 * lr; cursor 0.  dev: caller's device memory, 256-byte aligned.  One copy on
 * `stream`, waited for: call it before capture.  Errors: ZS_ERR_NULL,
 * ZS_ERR_ARG, ZS_ERR_RANGE, ZS_ERR_CAPACITY, ZS_ERR_HIP, ZS_ERR_RESOURCE. */
zs_status zs_adamw_steps_init(const zs_adamw_hparams* hp, const double* lrs, int32_t nsteps,
                              void* dev, size_t bytes, void* stream, zs_adamw_steps* steps);

/* The next entry, as a one-wave kernel on `stream` (capturable).  sumsq: the
 * norm that the step was given, or NULL; where it is infinite or NaN the
 * cursor stays, so that a step that skip_nonfinite left out is not counted. */
zs_status zs_adamw_steps_advance(const zs_adamw_steps* steps, const double* sumsq, void* stream);

/* Reads the cursor and the exhausted flag back to the host (one copy on
 * `stream`, waited for). */
zs_status zs_adamw_steps_status(const zs_adamw_steps* steps, int64_t* cursor, int32_t* exhausted,
                                void* stream);

/* *sumsq = (accumulate ? *sumsq : 0) + the sum over all elements of the square
 * of the fp32 rank mean of the gradients, in double, in an order that is fixed
 * by the table and the device: the same bits every time.  store_mean: the fp32
 * mean also goes to every tensor's g_mean (with p > 1 a step that reads it
 * moves 8 bytes per element where reading the ranks again moves 2p).
 * accumulate continues a norm over several tables.
 * Bytes per element: p gradients, + 4 with store_mean.
 * Errors: ZS_ERR_NULL (also store_mean where a tensor has no g_mean),
 * ZS_ERR_ARG, ZS_ERR_DTYPE, ZS_ERR_ALIAS (sumsq lies in the table's
 * workspace), ZS_ERR_HIP. */
zs_status zs_grad_sumsq_multi(const zs_adamw_table* table, int32_t store_mean, int32_t accumulate,
                              double* sumsq, void* stream);

/* n fp32 moments to codes and scales (ceil(n / ZS_STATE8_BLOCK) of them),
 * rounded to nearest, and back (code times scale, fp32).  kind: ZS_STATE8_M
 * or ZS_STATE8_V (whose values are >= 0).  Bytes per value: 5.0156.
 * Errors: ZS_ERR_NULL, ZS_ERR_ARG, ZS_ERR_RANGE, ZS_ERR_ALIAS, ZS_ERR_HIP. */
zs_status zs_state8_encode(const float* x, int64_t n, int32_t kind, void* codes, float* scales,
                           void* stream);
zs_status zs_state8_decode(const void* codes, const float* scales, int64_t n, int32_t kind,
                           float* x, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ZSADAMW_H */
