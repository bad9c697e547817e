// zs_adamw.h -- the AdamW operators' launch descriptions (host and device).
#pragma once

#include "../../include/zsadamw.h"
#include "zs_internal.h"

namespace zs {

constexpr int kF32 = ZS_F32;
// A launch counts its lanes in 32 bits: 2^24 workgroups of 256 at most.
constexpr int64_t kMaxGroups = (int64_t{1} << 24) - 1;
constexpr int kStateBlock = ZS_STATE8_BLOCK;  // one wave: 64 lanes x 4 elements
constexpr int kUnit = 4 * kStateBlock;  // the shortest chunk, but for a tensor's last

// A run of at most chunk_elems elements of one tensor, with every address at
// its first element, so that a wave knows all it needs after one scalar load.
struct AwChunk {
  uint64_t w, m, v;           // addresses as numbers, see ld_chunk
  uint64_t m_scale, v_scale;
  uint64_t param;
  uint64_t g;                 // rank 0's gradient
  uint64_t g_mean;
  int64_t index;              // of element 0, for the random bits
  int64_t start;              // of element 0 in its tensor
  double lr_scale;
  double decay;
  int32_t len;
  int32_t piece;
  int64_t reserved[3];
};
static_assert(sizeof(AwChunk) == 128, "one table entry per 128-byte line");

// The scalars of one step, each computed in double and rounded once.
struct AwConsts {
  float B1, C1, B2, C2;
  float A1, A2;    // 1-beta1^t, 1-beta2^t (32-bit moments)
  float R2;        // 1/sqrt(1-beta2^t) (8-bit moments)
  float EPS;
  double inv_bc1;  // 1/(1-beta1^t) (8-bit moments)
  double lr;
  int64_t step;
};

// A step table on the device: launches that read it apply entry `cursor`; one
// that finds the cursor past the end does nothing and sets `exhausted`.
struct AwStepsDev {
  int64_t cursor;
  int64_t nsteps;
  int32_t exhausted;
  int32_t reserved[11];
  // nsteps AwConsts behind it
};
static_assert(sizeof(AwStepsDev) == 64, "the entries begin on a 64-byte boundary");

struct AwArgs {
  const AwChunk* chunks;
  const uint64_t* gptrs;     // npieces * p rank pointers at the tensors' first elements
  const double* sumsq;       // or null
  AwStepsDev* steps;         // or null: the constants below
  double grad_scale, max_norm;
  uint64_t seed;
  int32_t p;
  int32_t skip_nonfinite;
  int32_t shift;  // workgroups per chunk, a power of two's exponent
  float PF;       // f32(p)
  AwConsts c;
};

constexpr int log2_of(int x) { return x <= 1 ? 0 : 1 + log2_of(x / 2); }

struct AwLaunch {
  AwArgs a;
  int64_t nchunks;
  int log_blocks;  // blocks of 256 elements per chunk, a power of two's exponent
  int gdt, pdt, rounding;
  bool on_lines;  // every tensor's arrays begin on a 128-byte line
  hipStream_t stream;
};

struct SumsqLaunch {
  const AwChunk* chunks;
  const uint64_t* gptrs;
  int64_t nchunks;
  int log_blocks;  // as in AwLaunch
  int p, gdt;
  bool store, accumulate;
  double* partial;         // kSumsqBlocks doubles
  unsigned int* arrived;   // 0 between launches
  double* out;
  hipStream_t stream;
};
constexpr int kSumsqBlocks = 2048;  // workgroups of a sum of squares at most

hipError_t launch_adamw32(const AwLaunch& a);
hipError_t launch_adamw8(const AwLaunch& a);
hipError_t launch_sumsq(const SumsqLaunch& a);
// cursor += 1, unless sumsq is given and not finite.
hipError_t launch_steps_advance(AwStepsDev* t, const double* sumsq, hipStream_t stream);
hipError_t launch_state8_encode(const float* x, int64_t n, int kind, void* codes, float* scales,
                                hipStream_t stream);
hipError_t launch_state8_decode(const void* codes, const float* scales, int64_t n, int kind,
                                float* x, hipStream_t stream);

}  // namespace zs
