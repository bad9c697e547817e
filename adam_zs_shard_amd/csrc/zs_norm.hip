// zs_norm.hip -- layer norm and root-mean-square norm, forward (backward:
// zs_norm_grad.hip).
//
// Both passes stream: the forward pass reads and writes each row once, the
// backward pass reads two (or three) rows and writes one, at about 10 and 20 fp32
// operations per element, so HBM bounds them where rows are wide and many (16384 x
// 4096 bf16: forward with a residual 85.7 us, 6.3 TB/s; backward 88.5, 6.1, and 4.8
// for the second launch), and latency where they are narrow (8192 x 768: 7.3 and 15
// us) or few.  A row stays in the registers of a team of lanes from its only load to
// its store, so a team has 16 to 1024 lanes by the row's length, and the sums over
// it are sums over the team: DPP adds in a wave, LDS between waves.  The variance is
// the sum of squares of what remains after the mean is taken off, not the difference
// of two sums, which loses its digits where the mean is large.

#include "zs_norm_device.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

struct NormArgs {
  Rows x, residual, total, y;
  const void* gamma;
  const void* beta;
  float* mean;
  float* rstd;
  int64_t rows;
  int cols, wdt;
  float eps;
};

template <int DT, int TEAM, int J, bool WHOLE, bool STREAM>
__device__ __forceinline__ void ld_row(const Rows& rows, int64_t r, int lane, int cols, Pack<DT> (&q)[J]) {
  const char* at = reinterpret_cast<const char*>(rows.at + r * rows.pitch);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = (lane + j * TEAM) * kPack<DT>;
    q[j] = ld_some<DT, WHOLE, STREAM>(at, c, cols);
  }
}

template <int DT, int TEAM, int E, int WG, bool LAYER, bool WHOLE, bool STREAM>
__global__ __launch_bounds__(WG) void norm_kernel(NormArgs a) {
  constexpr int V = kPack<DT>, J = E / V, TEAMS = WG / TEAM;
  __shared__ float part[2][1][16];
  int turn = 0;
  const int lane = threadIdx.x % TEAM;
  const int team = team_of<TEAM>();
  Vals<V> gamma[J], beta[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = (lane + j * TEAM) * V;
    gamma[j] = ld_weights<V>(a.gamma, a.wdt, c, a.cols, 1.0f);
    beta[j] = ld_weights<V>(a.beta, a.wdt, c, a.cols, 0.0f);
  }
  const float n = static_cast<float>(a.cols);
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * TEAMS; r0 < a.rows;
       r0 += static_cast<int64_t>(gridDim.x) * TEAMS) {
    const int64_t r = r0 + team;
    if (TEAMS > 1 && r >= a.rows) return;  // such a team waits for nobody
    float t[J][V];
    Pack<DT> q[J];
    ld_row<DT, TEAM, J, WHOLE, STREAM>(a.x, r, lane, a.cols, q);
    Pack<DT> p[J];
    if (a.residual.at) ld_row<DT, TEAM, J, WHOLE, STREAM>(a.residual, r, lane, a.cols, p);
#pragma unroll
    for (int j = 0; j < J; ++j) settle<DT, WHOLE>(q[j], (lane + j * TEAM) * V, a.cols);
    if (a.residual.at) {
      char* total = reinterpret_cast<char*>(a.total.at + r * a.total.pitch);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int c = (lane + j * TEAM) * V;
        float f[V];
        settle<DT, WHOLE>(p[j], c, a.cols);
        widen<DT>(q[j], t[j]);
        widen<DT>(p[j], f);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = t[j][i] + f[i];
        q[j] = narrow<DT>(f);
        st_some<DT, WHOLE>(total + c * kSize<DT>, a.cols - c, q[j]);
      }
    }
    float mean = 0.0f;
    if constexpr (LAYER) {
      float s[1] = {0.0f};
#pragma unroll
      for (int j = 0; j < J; ++j) {
        widen<DT>(q[j], t[j]);
#pragma unroll
        for (int i = 0; i < V; ++i) s[0] += t[j][i];
      }
      team_sums<TEAM>(s, part, turn);
      mean = s[0] / n;
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int left = a.cols - (lane + j * TEAM) * V;
      widen<DT>(q[j], t[j]);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (LAYER) t[j][i] = (WHOLE ? left > 0 : i < left) ? t[j][i] - mean : 0.0f;
        s[0] = __builtin_fmaf(t[j][i], t[j][i], s[0]);
      }
    }
    team_sums<TEAM>(s, part, turn);
    const float rstd = 1.0f / __builtin_sqrtf(s[0] / n + a.eps);
    char* y = reinterpret_cast<char*>(a.y.at + r * a.y.pitch);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = (lane + j * TEAM) * V;
      float f[V];
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = (t[j][i] * rstd) * gamma[j].v[i] + beta[j].v[i];
      st_some<DT, WHOLE>(y + c * kSize<DT>, a.cols - c, narrow<DT>(f));
    }
    if (lane == 0) {
      if (LAYER && a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
}

// Workgroups of the forward pass: with a residual one row per team, which ends
// (16384 x 4096 bf16 85.9 us, 6.2 TB/s; 92.9 with 1024 lanes per CU that go on to
// further rows); without one, and for rows of 1024 lanes, as many elements per CU
// at a time (16384 x 4096 bf16, layer norm 47.8 us, one row per team 52.0; 4096 x
// 16384 56.9 and 70.9).
constexpr int kNormHeld = 16384;
// Where a call reads and writes more than this, its rows do not stay in the 256 MB
// cache from one kernel of a model to the next, and it reads past that (16384 x 4096
// with a residual 85.9 us, 89.8 read through it); smaller ones may have been left
// there by the kernel before (32768 x 1024 bf16 22.4 us, read past it 27.4).  Rows of
// broken packs are read through it at any size, since it makes no difference there:
// 40,000 x 1001 with a residual 63.8 us, past it 62.3, 16384 x 4099 154 and 154, 60,000
// x 1001 without one 50.4 and 50.8.
constexpr int64_t kNormCached = int64_t{192} << 20;

constexpr int norm_group(int team) { return team <= kWave ? 4 * kWave : team; }

}  // namespace

hipError_t launch_norm(const NormLaunch& L) {
  NormArgs a;
  a.x = L.x;
  a.residual = L.residual;
  a.total = L.total;
  a.y = L.y;
  a.gamma = L.gamma;
  a.beta = L.beta;
  a.mean = L.mean;
  a.rstd = L.rstd;
  a.rows = L.rows;
  a.cols = L.cols;
  a.wdt = L.wdt;
  a.eps = L.eps;
  const bool stream = L.rows * L.cols * (L.dt == kF32 ? 4 : 2) * (L.residual.at ? 4 : 2) > kNormCached;
  with_shape<16>(L.dt, L.cols, [&](auto d, auto team, auto e) {
    constexpr int TEAM = decltype(team)::value, WG = norm_group(TEAM), TEAMS = WG / TEAM;
    const int64_t groups = (L.rows + TEAMS - 1) / TEAMS;
    constexpr int64_t kMost = kMaxGroups / (WG > kBlock ? WG / kBlock : 1);
    constexpr int kPerCu = kNormHeld / decltype(e)::value / WG;
    const int64_t most = L.residual.at && TEAM < 1024 ? kMost : int64_t{cu_count()} * kPerCu;
    const dim3 grid(static_cast<unsigned>(groups < most ? groups : most));
    const auto go = [&](auto layer, auto whole, auto past) {
      norm_kernel<decltype(d)::value, TEAM, decltype(e)::value, WG, decltype(layer)::value != 0,
                  decltype(whole)::value != 0, decltype(past)::value != 0><<<grid, WG, 0, L.stream>>>(a);
    };
    const auto pick = [&](auto whole, auto past) {
      L.layer ? go(IC<1>{}, whole, past) : go(IC<0>{}, whole, past);
    };
    if (L.cols % kPack<decltype(d)::value> != 0) pick(IC<0>{}, IC<0>{});
    else if (stream) pick(IC<1>{}, IC<1>{});
    else pick(IC<1>{}, IC<0>{});
  });
  return hipGetLastError();
}

}  // namespace zs
