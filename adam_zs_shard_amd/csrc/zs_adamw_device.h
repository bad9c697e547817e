// zs_adamw_device.h -- device code shared by the AdamW kernels of libzshard.
//
// The AdamW step streams: per element p gradients, the fp32 master weight and
// the two moments in, the weight, the moments and the 16-bit copy out, and
// about 50 fp32 operations, so HBM bounds it (28 bytes per element with one
// bf16 gradient and 32-bit moments, 16.06 with 8-bit ones).  The unit is a
// block of 256 elements and one wave: lane l holds elements 4l .. 4l+3, so
// each access is one whole-line stream (fp32 1 KiB, 16-bit 512 bytes, codes
// 256 bytes per instruction), the largest value of an 8-bit block is one
// reduction over the wave, and no wave waits for another.
//
// Times in these files' comments are of one pass among many in a row on the GPU,
// over input sets that take turns.
#pragma once

#include "zs_adamw.h"
#include "zs_device.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

constexpr int kQuad = 4;
constexpr int kWave = 64;
constexpr int kWaves = kBlock / kWave;

// Codes may sit at any byte address.
typedef uint32_t u32b __attribute__((aligned(1)));

// An address out of a table, as one in global memory: the compiler cannot
// know that of a pointer that it loads, and accesses through a generic one
// (flat) make every wait a full drain.
template <class T>
__device__ __forceinline__ T* in_global(uint64_t x) {
  using GT = __attribute__((address_space(1))) T;
  return (T*)reinterpret_cast<GT*>(x);
}
struct Chunk {
  float* w;
  char* m;
  char* v;
  float* m_scale;
  float* v_scale;
  uint16_t* param;
  const char* g;
  float* g_mean;
  int64_t index, start;
  double lr_scale, decay;
  int32_t len, piece;
};
__device__ __forceinline__ Chunk ld_chunk(const AwChunk* at) {
  const AwChunk& c = *at;
  return Chunk{in_global<float>(c.w),        in_global<char>(c.m),
               in_global<char>(c.v),         in_global<float>(c.m_scale),
               in_global<float>(c.v_scale),  in_global<uint16_t>(c.param),
               in_global<const char>(c.g),   in_global<float>(c.g_mean),
               c.index, c.start, c.lr_scale, c.decay, c.len, c.piece};
}

template <class F>
void with_gdt(int dt, F&& f) {
  if (dt == kF16) f(IC<kF16>{});
  else if (dt == kBF16) f(IC<kBF16>{});
  else f(IC<kF32>{});
}

// ---- four elements of a lane ------------------------------------------------
template <int DT>
struct Raw4 {
  u32x2 x;
};
template <>
struct Raw4<kF32> {
  f32x4 x;
};

template <int DT>
constexpr int kSize = DT == kF32 ? 4 : 2;

// Non-temporal unless STREAM is false.
template <int DT, bool STREAM = true>
__device__ __forceinline__ Raw4<DT> ld_raw4(const void* base, uint32_t lane) {
  using T = std::conditional_t<DT == kF32, f32x4, u32x2>;
  const T* p = reinterpret_cast<const T*>(static_cast<const char*>(base) +
                                          lane * (kQuad * kSize<DT>));
  return Raw4<DT>{STREAM ? __builtin_nontemporal_load(p) : *p};
}
// The first n (0..4) of the lane's elements, zeros behind them.
template <int DT>
__device__ __forceinline__ Raw4<DT> ld_raw4(const void* base, uint32_t lane, int n) {
  if constexpr (DT == kF32) {
    const float* p = static_cast<const float*>(base) + lane * kQuad;
    f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < kQuad; ++j)
      if (j < n) x[j] = p[j];
    return Raw4<DT>{x};
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + lane * kQuad;
    uint32_t h[kQuad] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < kQuad; ++j)
      if (j < n) h[j] = p[j];
    return Raw4<DT>{u32x2{h[0] | h[1] << 16, h[2] | h[3] << 16}};
  }
}

template <int DT>
__device__ __forceinline__ void widen4(const Raw4<DT>& q, float (&x)[kQuad]) {
  if constexpr (DT == kF32) {
#pragma unroll
    for (int j = 0; j < kQuad; ++j) x[j] = q.x[j];
  } else {
    x[0] = widen_lo<DT>(q.x[0]);
    x[1] = widen_hi<DT>(q.x[0]);
    x[2] = widen_lo<DT>(q.x[1]);
    x[3] = widen_hi<DT>(q.x[1]);
  }
}

__device__ __forceinline__ void st_quad32(float* base, uint32_t lane, const float (&x)[kQuad]) {
  __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]},
                              reinterpret_cast<f32x4*>(base + lane * kQuad));
}
__device__ __forceinline__ void st_quad32(float* base, uint32_t lane, int n,
                                          const float (&x)[kQuad]) {
#pragma unroll
  for (int j = 0; j < kQuad; ++j)
    if (j < n) base[lane * kQuad + j] = x[j];
}
template <int DT>
__device__ __forceinline__ void st_quad16(uint16_t* base, uint32_t lane, const float (&x)[kQuad]) {
  __builtin_nontemporal_store(u32x2{narrow2<DT>(x[0], x[1]), narrow2<DT>(x[2], x[3])},
                              reinterpret_cast<u32x2*>(base + lane * kQuad));
}
template <int DT>
__device__ __forceinline__ void st_quad16(uint16_t* base, uint32_t lane, int n,
                                          const float (&x)[kQuad]) {
#pragma unroll
  for (int j = 0; j < kQuad; ++j)
    if (j < n) base[lane * kQuad + j] = narrow1<DT>(x[j]);
}
// Four codes, one per byte.  Plain loads: a wave's 256 bytes of codes that do
// not begin on a line share theirs with the next wave's, which non-temporal
// loads fetch twice (4.0e8 elements in buffers 3 elements into a line 1.12 ms,
// non-temporal 1.24; on a line 1.01, 1.04).
__device__ __forceinline__ uint32_t ld_codes(const void* base, uint32_t lane) {
  return *reinterpret_cast<const u32b*>(static_cast<const char*>(base) + lane * kQuad);
}
__device__ __forceinline__ uint32_t ld_codes(const void* base, uint32_t lane, int n) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + lane * kQuad;
  uint32_t x = 0;
#pragma unroll
  for (int j = 0; j < kQuad; ++j)
    if (j < n) x |= static_cast<uint32_t>(p[j]) << (8 * j);
  return x;
}
__device__ __forceinline__ void st_codes(void* base, uint32_t lane, uint32_t x) {
  __builtin_nontemporal_store(
      x, reinterpret_cast<u32b*>(static_cast<char*>(base) + lane * kQuad));
}
__device__ __forceinline__ void st_codes(void* base, uint32_t lane, int n, uint32_t x) {
  uint8_t* p = static_cast<uint8_t*>(base) + lane * kQuad;
#pragma unroll
  for (int j = 0; j < kQuad; ++j)
    if (j < n) p[j] = static_cast<uint8_t>(x >> (8 * j));
}

// ---- gradients ----------------------------------------------------------------
typedef const uint64_t __attribute__((address_space(4)))* RankPtrs;
__device__ __forceinline__ RankPtrs rank_ptrs(const uint64_t* gptrs, int piece, int p) {
  return (RankPtrs)(reinterpret_cast<uintptr_t>(gptrs + static_cast<int64_t>(piece) * p));
}

// Loads of R ranks' shares of a block in flight together, then the adds in
// rank order.  n < 0: a whole block; else the lane's first n (0..4) elements.
template <int R, int GDT>
__device__ __forceinline__ void add_ranks(RankPtrs ptrs, int r0, int64_t byte0, uint32_t lane,
                                          int n, float (&s)[kQuad]) {
  Raw4<GDT> q[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const char* base = in_global<const char>(ptrs[r0 + r]) + byte0;
    q[r] = n < 0 ? ld_raw4<GDT>(base, lane) : ld_raw4<GDT>(base, lane, n);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float x[kQuad];
    widen4<GDT>(q[r], x);
#pragma unroll
    for (int j = 0; j < kQuad; ++j) s[j] = r0 + r == 0 ? x[j] : s[j] + x[j];
  }
}

// The rank-order mean of the block that starts `at` elements into its tensor.
// Eight ranks' loads at a time: 15.6M elements, 8 ranks, 32-bit moments 106 us
// against 109 with four; 30M and 16 ranks 277 against 314.
template <int GDT>
__device__ __forceinline__ void mean_ranks(RankPtrs ptrs, int p, float PF, int64_t at,
                                           uint32_t lane, int n, float (&s)[kQuad]) {
  const int64_t byte0 = at * kSize<GDT>;
  int r = 0;
  for (; r + 8 <= p; r += 8) add_ranks<8, GDT>(ptrs, r, byte0, lane, n, s);
  if (r + 4 <= p) {
    add_ranks<4, GDT>(ptrs, r, byte0, lane, n, s);
    r += 4;
  }
  if (r + 2 <= p) {
    add_ranks<2, GDT>(ptrs, r, byte0, lane, n, s);
    r += 2;
  }
  if (r < p) add_ranks<1, GDT>(ptrs, r, byte0, lane, n, s);
#pragma unroll
  for (int j = 0; j < kQuad; ++j) s[j] = s[j] / PF;
}

// ---- 8-bit moments ------------------------------------------------------------
constexpr float kTopM = 448.0f, kTopV = 57344.0f;
constexpr uint32_t kTinyBits = (127u - 110u) << 23;  // 2^-110
constexpr uint32_t kInfBits = 0x7f800000u;

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
  const uint32_t y = static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, 0xf, 0xf, true));
  return x > y ? x : y;
}

// The largest of the wave's values (fp32 magnitudes compare as their bits,
// NaN above infinity above the rest).  Every lane must be active.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = dpp_max<0xb1>(x);   // lanes xor 1
  x = dpp_max<0x4e>(x);   // xor 2
  x = dpp_max<0x141>(x);  // mirrored in eights
  x = dpp_max<0x140>(x);  // mirrored in sixteens
  const uint32_t a = __builtin_amdgcn_readlane(x, 0), b = __builtin_amdgcn_readlane(x, 16);
  const uint32_t c = __builtin_amdgcn_readlane(x, 32), d = __builtin_amdgcn_readlane(x, 48);
  const uint32_t ab = a > b ? a : b, cd = c > d ? c : d;
  return ab > cd ? ab : cd;
}

__device__ __forceinline__ uint32_t mag_bits(float x) {
  return __float_as_uint(x) & 0x7fffffffu;
}

template <int KIND>
constexpr float kTop = KIND == ZS_STATE8_M ? kTopM : kTopV;
template <int KIND>  // the smallest normal code
constexpr float kLeast = KIND == ZS_STATE8_M ? 0x1p-6f : 0x1p-14f;

// One over the type's largest value, rounded once.
template <int KIND>
constexpr float kDown = static_cast<float>(1.0 / static_cast<double>(kTop<KIND>));

// A block's largest value, of its magnitudes' bits: what becomes of it.
struct BlockScale {
  float scale;    // stored
  float inverse;  // the values' factor before they are rounded
  bool codes;     // neither a block of zeros nor one that is not finite
};

template <int KIND>
__device__ __forceinline__ BlockScale block_scale(uint32_t most) {
  BlockScale s{0.0f, 0.0f, most >= kTinyBits && most < kInfBits};
  if (most >= kTinyBits) {
    s.scale = __uint_as_float(most) * kDown<KIND>;
    s.inverse = kTop<KIND> / __uint_as_float(most);
  }
  if (most >= kInfBits) s.scale = __uint_as_float(0x7fc00000u);
  return s;
}

// Both moments' scales with one division: lanes 0..31 work on m, the others
// on v.  `mine` is the lane's half's stored scale.
__device__ __forceinline__ void block_scales(uint32_t mm, uint32_t vm, uint32_t lane,
                                             BlockScale& sm, BlockScale& sv, float& mine) {
  const bool hi = lane >= kWave / 2;
  const uint32_t most = hi ? vm : mm;
  const float inverse = (hi ? kTopV : kTopM) / __uint_as_float(most);
  const float scale = __uint_as_float(most) * (hi ? kDown<ZS_STATE8_V> : kDown<ZS_STATE8_M>);
  mine = most >= kInfBits ? __uint_as_float(0x7fc00000u) : most >= kTinyBits ? scale : 0.0f;
  sm.inverse = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(inverse), 0));
  sv.inverse = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(inverse), kWave / 2));
  sm.codes = mm >= kTinyBits && mm < kInfBits;
  sv.codes = vm >= kTinyBits && vm < kInfBits;
}

template <int KIND>
__device__ __forceinline__ uint32_t pack4(const float (&y)[kQuad]) {
  int c = 0;
  if constexpr (KIND == ZS_STATE8_M) {
    c = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], c, false);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], c, true);
  } else {
    c = __builtin_amdgcn_cvt_pk_bf8_f32(y[0], y[1], c, false);
    c = __builtin_amdgcn_cvt_pk_bf8_f32(y[2], y[3], c, true);
  }
  return static_cast<uint32_t>(c);
}

// Random rounding of a magnitude that may lie on the even part of the grid.
template <int KIND>
__device__ __forceinline__ float to_grid(float y, uint32_t half) {
  constexpr int kCut = KIND == ZS_STATE8_M ? 20 : 21;
  const float mag = __builtin_fabsf(y);
  const bool low = mag < kLeast<KIND>;
  const float up = low ? mag + kLeast<KIND> : mag;
  const uint32_t r = (half << (kCut - 16)) + (1u << (kCut - 17));
  const float cut = __uint_as_float((__float_as_uint(up) + r) & ~((1u << kCut) - 1u));
  return __builtin_copysignf(low ? cut - kLeast<KIND> : cut, y);
}

// Four values to codes: x * inverse cut to [-top, top], to the nearest code or
// by the random halves (m: the words' low 16 bits, v: the high ones), a
// positive v never to code 0.  Every lane must be active.  The hardware's
// random rounding (v_cvt_sr) adds its bits to a normal value's fraction and
// cuts, which is the definition with the half above and a single bit below
// it; for values on the even part of the grid, and v's that might get code 0, a
// wave takes the longer way.  Gaussian moments of one size have such values in
// about 2% of the waves; 4.0e8 elements take 1.01 ms then, and the same with an
// outlier in every block, or with half the moments zero: HBM hides it.
template <int KIND, bool RANDOM>
__device__ __forceinline__ uint32_t encode4(const float (&x)[kQuad], const BlockScale& s,
                                            const uint32_t (&word)[kQuad]) {
  if (!s.codes) return 0u;
  constexpr float top = kTop<KIND>;
  float y[kQuad];
#pragma unroll
  for (int j = 0; j < kQuad; ++j)
    y[j] = __builtin_fminf(__builtin_fmaxf(x[j] * s.inverse, -top), top);
  if constexpr (!RANDOM && KIND == ZS_STATE8_M) return pack4<KIND>(y);
  const float least =
      __builtin_fminf(__builtin_fminf(__builtin_fabsf(y[0]), __builtin_fabsf(y[1])),
                      __builtin_fminf(__builtin_fabsf(y[2]), __builtin_fabsf(y[3])));
  const bool special = __builtin_amdgcn_ballot_w64(least < kLeast<KIND>) != 0;
  if (!special) {
    if constexpr (!RANDOM) return pack4<KIND>(y);
    int c = 0;
    if constexpr (KIND == ZS_STATE8_M) {
      c = __builtin_amdgcn_cvt_sr_fp8_f32(y[0], (word[0] << 16) | 0x8000u, c, 0);
      c = __builtin_amdgcn_cvt_sr_fp8_f32(y[1], (word[1] << 16) | 0x8000u, c, 1);
      c = __builtin_amdgcn_cvt_sr_fp8_f32(y[2], (word[2] << 16) | 0x8000u, c, 2);
      c = __builtin_amdgcn_cvt_sr_fp8_f32(y[3], (word[3] << 16) | 0x8000u, c, 3);
    } else {
      c = __builtin_amdgcn_cvt_sr_bf8_f32(y[0], (word[0] & 0xffff0000u) | 0x8000u, c, 0);
      c = __builtin_amdgcn_cvt_sr_bf8_f32(y[1], (word[1] & 0xffff0000u) | 0x8000u, c, 1);
      c = __builtin_amdgcn_cvt_sr_bf8_f32(y[2], (word[2] & 0xffff0000u) | 0x8000u, c, 2);
      c = __builtin_amdgcn_cvt_sr_bf8_f32(y[3], (word[3] & 0xffff0000u) | 0x8000u, c, 3);
    }
    return static_cast<uint32_t>(c);
  }
  if constexpr (RANDOM) {
#pragma unroll
    for (int j = 0; j < kQuad; ++j)
      y[j] = to_grid<KIND>(y[j], KIND == ZS_STATE8_M ? word[j] & 0xffffu : word[j] >> 16);
  }
  uint32_t u = pack4<KIND>(y);
  if constexpr (KIND == ZS_STATE8_V) {
#pragma unroll
    for (int j = 0; j < kQuad; ++j)
      if (x[j] > 0.0f && ((u >> (8 * j)) & 0xffu) == 0u) u |= 1u << (8 * j);
  }
  return u;
}

template <int KIND>
__device__ __forceinline__ void decode4(uint32_t c, float scale, float (&x)[kQuad]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  f32x2 a, b;
  if constexpr (KIND == ZS_STATE8_M) {
    a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c), false);
    b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c), true);
  } else {
    a = __builtin_amdgcn_cvt_pk_f32_bf8(static_cast<int>(c), false);
    b = __builtin_amdgcn_cvt_pk_f32_bf8(static_cast<int>(c), true);
  }
  x[0] = a[0] * scale;
  x[1] = a[1] * scale;
  x[2] = b[0] * scale;
  x[3] = b[1] * scale;
}

// Philox4x32 with 7 rounds (Salmon et al., SC'11): four random words from a
// counter and a key.
__device__ __forceinline__ void philox(uint64_t at, uint64_t step, uint64_t seed,
                                       uint32_t (&w)[kQuad]) {
  uint32_t c0 = static_cast<uint32_t>(at), c1 = static_cast<uint32_t>(at >> 32);
  uint32_t c2 = static_cast<uint32_t>(step), c3 = static_cast<uint32_t>(step >> 32);
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u;
    const uint64_t b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = __builtin_amdgcn_bitop3_b32(static_cast<uint32_t>(b >> 32), c1, k0, 0x96);  // xor
    c1 = static_cast<uint32_t>(b);
    c2 = __builtin_amdgcn_bitop3_b32(static_cast<uint32_t>(a >> 32), c3, k1, 0x96);
    c3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  w[0] = c0;
  w[1] = c1;
  w[2] = c2;
  w[3] = c3;
}

// ---- the step's scalars -------------------------------------------------------
struct Scalars {
  float GS;   // the gradient's factor
  bool skip;  // the norm is not finite and such a step is to be left out
};

__device__ __forceinline__ Scalars scalars(const AwArgs& a) {
  if (!a.sumsq) return Scalars{static_cast<float>(a.grad_scale), false};
  const double sumsq = *a.sumsq;
  double coef = 1.0;
  if (a.max_norm > 0.0) {
    coef = a.max_norm / (__builtin_sqrt(sumsq) * __builtin_fabs(a.grad_scale) + 1e-6);
    coef = coef > 1.0 ? 1.0 : coef;  // NaN stays
  }
  return Scalars{static_cast<float>(a.grad_scale * coef),
                 a.skip_nonfinite != 0 && !__builtin_isfinite(sumsq)};
}

// One element's moments, in the order of the fp32 definition.
__device__ __forceinline__ void moments1(const AwConsts& c, float g, float& m, float& v) {
  m = c.B1 * m + c.C1 * g;
  v = c.B2 * v + c.C2 * (g * g);
}

}  // namespace
}  // namespace zs
