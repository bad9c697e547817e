// zs_layer.h -- the layer operators' launch descriptions (host and device).
#pragma once

#include "../../include/zslayer.h"
#include "zs_adamw.h"

namespace zs {

// Rows of activations: the first element's address and the bytes between rows.
struct Rows {
  uintptr_t at;
  int64_t pitch;
};

struct NormLaunch {
  int64_t rows;
  int cols;
  int dt, wdt;
  bool layer;
  float eps;
  Rows x, residual, total, y;  // residual.at 0: none
  const void* gamma;           // or null
  const void* beta;            // or null
  float* mean;                 // or null
  float* rstd;                 // or null
  hipStream_t stream;
};
hipError_t launch_norm(const NormLaunch& L);

// Workgroups of the norm's backward pass at most, each with one row of partial
// sums per gradient in the workspace.
constexpr int kNormParts = 512;
// Columns of such a row at most: what the lanes of a team hold, 8 or 16 columns each.
constexpr int norm_width(int cols) {
  int width = 512;
  while (width < cols) width *= 2;
  return width;
}

struct NormGradLaunch {
  int64_t rows;
  int cols;
  int dt, wdt, gdt;
  bool layer, accumulate;
  Rows dy, x, dres, dx;  // dres.at 0: none
  const void* gamma;     // or null
  const float* mean;
  const float* rstd;
  void* dgamma;          // or null
  void* dbeta;           // or null
  float* partial;        // kNormParts rows of norm_width of dgamma's sums, then of dbeta's
  hipStream_t stream;
};
hipError_t launch_norm_grad(const NormGradLaunch& L);

struct EmbedLaunch {
  int64_t tokens, rows, first_row, pos_rows;
  int cols;
  int dt, tdt;
  bool wide_ids;  // 64-bit
  float scale;
  const void* ids;
  const void* table;
  const void* pos_ids;
  const void* pos_table;  // or null
  Rows y;
  hipStream_t stream;
};
hipError_t launch_embed(const EmbedLaunch& L);

// A token and the row of the table that it names (the table's number of rows:
// none).
struct TokenRow {
  uint32_t row, token;
};

// Where the parts of an embedding gradient's workspace lie.
struct EmbedLayout {
  size_t list;       // the tokens in the order of their rows
  size_t other;      // the same before or after a pass of the sort
  size_t counts;     // of a pass's digits, per tile of the tokens
  size_t long_rows;  // rows whose tokens are summed in parts
  size_t partial;    // these parts
  size_t total;
};
// Tokens that are sorted in one launch at most, and the bits of a digit at most,
// in that launch and in several.
constexpr int64_t kSortAlone = 16384;
constexpr int kBucketBits = 8, kSortBits = 10;
EmbedLayout embed_layout(int64_t tokens, int64_t cols);
// The most that a call of so many tokens (>= 1) or fewer takes.
size_t embed_workspace(int64_t tokens, int64_t cols);

struct EmbedGradLaunch {
  int64_t tokens, rows, first_row;
  int cols;
  int dt, gdt;
  bool wide_ids, accumulate;
  float scale;
  const void* ids;
  Rows dy;
  void* grad;
  unsigned char* workspace;
  hipStream_t stream;
};
hipError_t launch_embed_grad(const EmbedGradLaunch& L);

}  // namespace zs
