// zs_norm_device.h -- what the norms' forward and backward kernels share: teams of
// lanes that hold a row.
#pragma once

#include "zs_layer_device.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

// A team's number in its workgroup: the same for a wave's lanes, unless several teams
// share it.
template <int TEAM>
__device__ __forceinline__ int team_of() {
  const int team = threadIdx.x / TEAM;
  return TEAM < kWave ? team : __builtin_amdgcn_readfirstlane(team);
}

// The sum over a team's lanes, in every one of them.  Between waves it goes
// through part, two of which take turns, so that one barrier per sum will do:
// who writes part k again has passed the barrier of part k + 1, before which
// every wave has read part k.
template <int TEAM, int N>
__device__ __forceinline__ void team_sums(float (&x)[N], float (*part)[N][16], int& turn) {
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = lanes_sum<(TEAM < kWave ? TEAM : kWave)>(x[k]);
  if constexpr (TEAM > kWave) {
    constexpr int W = TEAM / kWave;
    const int wave = threadIdx.x / kWave, first = wave / W * W;
    if (threadIdx.x % kWave == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) part[turn][k][wave] = x[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float s = part[turn][k][first];
#pragma unroll
      for (int i = 1; i < W; ++i) s += part[turn][k][first + i];
      x[k] = s;
    }
    turn ^= 1;
  }
}

// Calls f(dtype, team, elements per lane) for the smallest team that holds a row.
// A lane of the backward pass holds 8 elements (16 of the longest rows), so that
// its sums leave registers for 16 waves per CU.  The forward pass takes 16, half
// the waves per row (16384 x 4096 bf16, layer norm 47.8 us; 63.9 with 8).
// Teams of 16 and 32 lanes share a wave: a wave to each row is 262,144 x 128 bf16 rms
// forward 52.1 us for 22.3 and backward 75.2 for 37.2, 40,000 x 256 13.6 for 8.5 and
// 22.7 for 19.2.
// Teams double, so that rows between two sizes leave lanes without elements: layer
// norm, bf16, TB/s forward and backward, 8192 x 8192 5.7 and 4.6, 8192 x 5120 4.9 and
// 3.7, 8192 x 6144 4.8 and 3.9, 4096 x 12288 4.0 and 3.4, 16384 x 1280 4.5 and 3.4,
// 16384 x 1600 5.1 and 4.1, 16384 x 2560 5.2 and 3.8.
template <int E, class F>
void with_shape(int dt, int cols, F&& f) {
  with_gdt(dt, [&](auto d) {
    if (cols <= 16 * 8) f(d, IC<16>{}, IC<8>{});
    else if (cols <= 32 * 8) f(d, IC<32>{}, IC<8>{});
    else if (cols <= 64 * 8) f(d, IC<64>{}, IC<8>{});
    else if (cols <= 64 * E) f(d, IC<64>{}, IC<E>{});
    else if (cols <= 128 * E) f(d, IC<128>{}, IC<E>{});
    else if (cols <= 256 * E) f(d, IC<256>{}, IC<E>{});
    else if (cols <= 512 * E) f(d, IC<512>{}, IC<E>{});
    else if (cols <= 1024 * E) f(d, IC<1024>{}, IC<E>{});
    else f(d, IC<1024>{}, IC<16>{});
  });
}
static_assert(ZS_NORM_MAX_COLS == 1024 * 16, "the longest row is a team of 1024 lanes");

}  // namespace
}  // namespace zs
