// zs_adamw_norm.hip -- the sum of squares of the gradient mean, and moments to
// and from their 8-bit form.

#include "zs_adamw_device.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

// The sum of the values of a workgroup of W waves, in a fixed order.
template <int W>
__device__ __forceinline__ double block_sum(double x) {
  __shared__ double part[W];
#pragma unroll
  for (int d = kWave / 2; d > 0; d /= 2) x += __shfl_xor(x, d, kWave);
  if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = x;
  __syncthreads();
  double s = part[0];
#pragma unroll
  for (int i = 1; i < W; ++i) s += part[i];
  __syncthreads();
  return s;
}

template <int U, int GDT, bool STORE, bool ONE>
__device__ __forceinline__ void sumsq_blocks(const Chunk& ch, const uint64_t* gptrs, int p,
                                             float PF, int b, uint32_t lane, int n, double& acc) {
  const int64_t e0 = static_cast<int64_t>(b) * kStateBlock;
  float g[U][kQuad];
  if constexpr (ONE) {
    Raw4<GDT> q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const char* gb = ch.g + (e0 + u * kStateBlock) * kSize<GDT>;
      q[u] = n < 0 ? ld_raw4<GDT>(gb, lane) : ld_raw4<GDT>(gb, lane, n);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) widen4<GDT>(q[u], g[u]);
  } else {
    static_assert(U == 1, "one block of several ranks at a time");
    mean_ranks<GDT>(rank_ptrs(gptrs, ch.piece, p), p, PF, ch.start + e0, lane, n, g[0]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if constexpr (STORE) {
      if (n < 0)
        st_quad32(ch.g_mean + e0 + u * kStateBlock, lane, g[u]);
      else
        st_quad32(ch.g_mean + e0 + u * kStateBlock, lane, n, g[u]);
    }
    // a product of two fp32 values is exact in double
#pragma unroll
    for (int j = 0; j < kQuad; ++j)
      acc = __builtin_fma(static_cast<double>(g[u][j]), static_cast<double>(g[u][j]), acc);
  }
}

// Joining the workgroups' sums.  JOIN: the last workgroup to arrive adds them
// up, in their order whoever it is, and makes the count ready for the next
// launch.  That saves a launch (3 us of the host's time), but each arrival
// writes back and invalidates its L2: with 1024 workgroups it cost 40 us (15.6M
// elements, 8 ranks: 62 -> 105 us).  So at most kJoinMost workgroups do it: of
// kJoinWaves waves each for one rank's sums of up to kJoinTurns turns of theirs
// (us on the GPU and on the host, against two launches: 50,000 elements 4.3 and
// 4.7, 5.0 and 7.8; 500,000 4.7 and 4.4, 5.0 and 7.0; 1.0e6 6.1 and 4.5, 5.3 and
// 6.9; with two more turns 2.0e6 8.5 and 4.4, 5.6 and 7.1; sixteen waves, once
// tried, took 0.9 more at 50,000), of four waves for several ranks' sums of one
// turn.
constexpr int kJoinMost = 64, kJoinWaves = 8, kJoinTurns = 2;

// One rank: four blocks per wave and turn, so that as many bytes are in
// flight, four workgroups per CU (1.0e9 bf16 elements in a graph's replays 299
// us, 6.7 TB/s, called in a row 285; replays with two, three and five 468 / 332
// / 297, eight blocks 332, two 467).  More ranks: one block of each, three
// workgroups per CU, so that the window swept at a time stays narrow (60M
// elements, 8 ranks, the mean kept: 198 us, 6.07 TB/s; two, four and five 230 /
// 206 / 224, eight and four blocks, once tried, 222 and 214).
constexpr int kLogOne = 2;
constexpr int kLoadsOne = 1 << kLogOne;
constexpr int kGroupsOne = 4, kGroupsRanks = 3;

// A unit is the U blocks that a wave of W takes at a turn; a chunk has 2^shift.
template <int W, int U, int GDT, bool STORE, bool ONE, bool JOIN>
__global__ __launch_bounds__(W * kWave) void sumsq_kernel(const AwChunk* chunks,
                                                          const uint64_t* gptrs, int64_t nunits,
                                                          int shift, int p, float PF,
                                                          double* partial, unsigned int* arrived,
                                                          int accumulate, double* out) {
  const uint32_t lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  double acc = 0.0;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * W + wave; i < nunits;
       i += static_cast<int64_t>(gridDim.x) * W) {
    const Chunk ch = ld_chunk(chunks + (i >> shift));
    const int b = static_cast<int>(i & ((1 << shift) - 1)) * U;
    const int left = ch.len - b * kStateBlock;
    if (left >= U * kStateBlock) {
      sumsq_blocks<U, GDT, STORE, ONE>(ch, gptrs, p, PF, b, lane, -1, acc);
      continue;
    }
    for (int k = 0; k < U && k * kStateBlock < left; ++k) {
      int n = left - k * kStateBlock - kQuad * static_cast<int>(lane);
      n = n < 0 ? 0 : n > kQuad ? kQuad : n;
      sumsq_blocks<1, GDT, STORE, ONE>(ch, gptrs, p, PF, b + k, lane, n, acc);
    }
  }
  const double s = block_sum<W>(acc);
  if constexpr (!JOIN) {
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
  } else {
    __shared__ bool last;
    if (threadIdx.x == 0) {
      __hip_atomic_store(partial + blockIdx.x, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = __hip_atomic_fetch_add(arrived, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
             gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    acc = 0.0;
    if (threadIdx.x < gridDim.x)
      acc = __hip_atomic_load(partial + threadIdx.x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const double total = block_sum<W>(acc);
    if (threadIdx.x == 0) {
      *out = accumulate ? *out + total : total;
      __hip_atomic_store(arrived, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
}
static_assert(kJoinMost <= kBlock, "one sum per thread in the join");

// One lane per sum on a card of 256 CUs (15.6M elements, 8 ranks 56.8 us in
// all; 57.0 with 256 lanes).
constexpr int kJoinLanes = 1024;

__global__ __launch_bounds__(kJoinLanes) void sumsq_join_kernel(const double* partial, int n,
                                                                int accumulate, double* out) {
  double acc = 0.0;
  for (int i = threadIdx.x; i < n; i += kJoinLanes) acc += partial[i];
  const double s = block_sum<kJoinLanes / kWave>(acc);
  if (threadIdx.x == 0) *out = accumulate ? *out + s : s;
}

__global__ void steps_advance_kernel(AwStepsDev* t, const double* sumsq) {
  if (threadIdx.x == 0 && (!sumsq || __builtin_isfinite(*sumsq))) t->cursor = t->cursor + 1;
}

// Conversions: a wave takes U blocks of 256 values, its loads first.  Two where
// there are enough for all CUs' waves: 117M values to 8 bits 93 us, 6.3 TB/s
// (one 102), from 8 bits 83 (81), 1.0e9 to 8 bits 789 us (841), from 8 bits 795
// (898); one below kConvertFew values.  Around it, us to / from 8 bits, two
// blocks 3.8 / 3.2 at 2.0e6, 5.4 / 4.5 at 4.0e6 and 9.2 / 7.1 at 8.0e6, one
// 3.4 / 3.2, 5.5 / 4.4 and 9.7 / 7.2; 50,000 values 2.2 / 2.8 and 1.9 / 2.1.
constexpr int kConvertWaves = 8;
constexpr int64_t kConvertFew = int64_t{1} << 21;

template <int U, int KIND>
__device__ __forceinline__ void encode_blocks(const float* x, uint8_t* codes, float* scales,
                                              int64_t b, uint32_t lane, int n) {
  Raw4<kF32> q[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float* at = x + (b + u) * kStateBlock;
    q[u] = n < 0 ? ld_raw4<kF32>(at, lane) : ld_raw4<kF32>(at, lane, n);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float y[kQuad];
    widen4<kF32>(q[u], y);
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < kQuad; ++j) most = mag_bits(y[j]) > most ? mag_bits(y[j]) : most;
    const BlockScale s = block_scale<KIND>(wave_max(most));
    const uint32_t none[kQuad] = {0u, 0u, 0u, 0u};
    const uint32_t c = encode4<KIND, false>(y, s, none);
    uint8_t* to = codes + (b + u) * kStateBlock;
    if (n < 0)
      st_codes(to, lane, c);
    else
      st_codes(to, lane, n, c);
    if (lane == 0) scales[b + u] = s.scale;
  }
}

template <int U, int KIND>
__device__ __forceinline__ void decode_blocks(const uint8_t* codes, const float* scales, float* x,
                                              int64_t b, uint32_t lane, int n) {
  uint32_t c[U];
  float s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint8_t* at = codes + (b + u) * kStateBlock;
    c[u] = n < 0 ? ld_codes(at, lane) : ld_codes(at, lane, n);
    s[u] = scales[b + u];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float y[kQuad];
    decode4<KIND>(c[u], s[u], y);
    float* to = x + (b + u) * kStateBlock;
    if (n < 0)
      st_quad32(to, lane, y);
    else
      st_quad32(to, lane, n, y);
  }
}

// Calls f(U blocks, first block, values of this lane or -1) for the wave's
// blocks of n values.
template <int U, class F>
__device__ __forceinline__ void convert_all(int64_t n, F&& f) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t whole = n / kStateBlock, blocks = (n + kStateBlock - 1) / kStateBlock;
  for (int64_t b = (static_cast<int64_t>(blockIdx.x) * kConvertWaves + wave) * U; b < blocks;
       b += static_cast<int64_t>(gridDim.x) * kConvertWaves * U) {
    if (b + U <= whole) {
      f(IC<U>{}, b, -1);
      continue;
    }
    for (int64_t k = b; k < b + U && k < blocks; ++k) {
      const int64_t left = n - k * kStateBlock - kQuad * static_cast<int>(threadIdx.x % kWave);
      f(IC<1>{}, k, left < 0 ? 0 : left > kQuad ? kQuad : static_cast<int>(left));
    }
  }
}

template <int U, int KIND>
__global__ __launch_bounds__(kConvertWaves * kWave) void encode_kernel(const float* x, int64_t n,
                                                                      uint8_t* codes,
                                                                      float* scales) {
  convert_all<U>(n, [&](auto u, int64_t b, int k) {
    encode_blocks<decltype(u)::value, KIND>(x, codes, scales, b, threadIdx.x % kWave, k);
  });
}

template <int U, int KIND>
__global__ __launch_bounds__(kConvertWaves * kWave) void decode_kernel(const uint8_t* codes,
                                                                      const float* scales,
                                                                      int64_t n, float* x) {
  convert_all<U>(n, [&](auto u, int64_t b, int k) {
    decode_blocks<decltype(u)::value, KIND>(codes, scales, x, b, threadIdx.x % kWave, k);
  });
}

// Calls f(U, KIND, workgroups): for all blocks of n values at once, up to what
// a launch counts.
template <class F>
void with_convert(int64_t n, int kind, F&& f) {
  const auto go = [&](auto u, auto k) {
    constexpr int64_t each = static_cast<int64_t>(decltype(u)::value) * kConvertWaves * kStateBlock;
    constexpr int64_t most = kMaxGroups * kBlock / (kConvertWaves * kWave);
    const int64_t groups = (n - 1) / each + 1;
    f(u, k, dim3(static_cast<unsigned>(groups < most ? groups : most)));
  };
  if (n < kConvertFew)
    kind == ZS_STATE8_M ? go(IC<1>{}, IC<ZS_STATE8_M>{}) : go(IC<1>{}, IC<ZS_STATE8_V>{});
  else
    kind == ZS_STATE8_M ? go(IC<2>{}, IC<ZS_STATE8_M>{}) : go(IC<2>{}, IC<ZS_STATE8_V>{});
}

}  // namespace

hipError_t launch_sumsq(const SumsqLaunch& L) {
  const bool one = L.p == 1;
  const int shift = one ? L.log_blocks - kLogOne : L.log_blocks;
  const int64_t nunits = L.nchunks << shift;
  const bool join = nunits <= kJoinMost * (one ? kJoinWaves * kJoinTurns : kWaves);
  const int waves = one && join ? kJoinWaves : kWaves;
  const int64_t most = join ? kJoinMost
                            : static_cast<int64_t>(cu_count()) * (one ? kGroupsOne : kGroupsRanks);
  int64_t grid = (nunits + waves - 1) / waves;
  if (grid > most) grid = most;
  if (grid > kSumsqBlocks) grid = kSumsqBlocks;
  if (grid < 1) grid = 1;  // no tensors: the sum is still written
  const float PF = static_cast<float>(static_cast<double>(L.p));
  with_gdt(L.gdt, [&](auto G) {
    constexpr int GDT = decltype(G)::value;
    const dim3 gd(static_cast<unsigned>(grid)), bd(static_cast<unsigned>(waves * kWave));
    const auto go = [&](auto w, auto u, auto store, auto join_) {
      constexpr int U = decltype(u)::value;
      sumsq_kernel<decltype(w)::value, U, GDT, decltype(store)::value != 0, U == kLoadsOne,
                   decltype(join_)::value != 0>
          <<<gd, bd, 0, L.stream>>>(L.chunks, L.gptrs, nunits, shift, L.p, PF, L.partial,
                                    L.arrived, L.accumulate ? 1 : 0, L.out);
    };
    const auto pick = [&](auto store) {
      if (one)
        join ? go(IC<kJoinWaves>{}, IC<kLoadsOne>{}, store, IC<1>{})
             : go(IC<kWaves>{}, IC<kLoadsOne>{}, store, IC<0>{});
      else
        join ? go(IC<kWaves>{}, IC<1>{}, store, IC<1>{}) : go(IC<kWaves>{}, IC<1>{}, store, IC<0>{});
    };
    L.store ? pick(IC<1>{}) : pick(IC<0>{});
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || join) return e;
  sumsq_join_kernel<<<dim3(1), dim3(kJoinLanes), 0, L.stream>>>(L.partial, static_cast<int>(grid),
                                                                L.accumulate ? 1 : 0, L.out);
  return hipGetLastError();
}

hipError_t launch_steps_advance(AwStepsDev* t, const double* sumsq, hipStream_t stream) {
  steps_advance_kernel<<<dim3(1), dim3(kWave), 0, stream>>>(t, sumsq);
  return hipGetLastError();
}

hipError_t launch_state8_encode(const float* x, int64_t n, int kind, void* codes, float* scales,
                                hipStream_t stream) {
  with_convert(n, kind, [&](auto u, auto k, dim3 grid) {
    encode_kernel<decltype(u)::value, decltype(k)::value>
        <<<grid, dim3(kConvertWaves * kWave), 0, stream>>>(x, n, static_cast<uint8_t*>(codes),
                                                           scales);
  });
  return hipGetLastError();
}

hipError_t launch_state8_decode(const void* codes, const float* scales, int64_t n, int kind,
                                float* x, hipStream_t stream) {
  with_convert(n, kind, [&](auto u, auto k, dim3 grid) {
    decode_kernel<decltype(u)::value, decltype(k)::value>
        <<<grid, dim3(kConvertWaves * kWave), 0, stream>>>(static_cast<const uint8_t*>(codes),
                                                           scales, n, x);
  });
  return hipGetLastError();
}

}  // namespace zs
