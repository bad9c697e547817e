// zs_norm.hip -- layer norm and root-mean-square norm, forward and backward.
//
// Both passes stream: the forward pass reads and writes each row once, the
// backward pass reads two (or three) rows and writes one, at about a dozen fp32
// operations per element, so HBM bounds them.  A row stays in the registers of
// a team of lanes from its only load to its store (16 elements per lane, so a
// team has 64 to 1024 lanes by the row's length), and the sums over it are sums
// over the team: DPP adds in a wave, LDS between waves.  The variance is the sum
// of squares of what remains after the mean is taken off, not the difference of
// two sums, which loses its digits where the mean is large.
//
// The weights' gradients are sums over rows.  Each lane keeps those of its own
// columns in registers over all rows that its team takes; the teams of a
// workgroup add theirs in LDS, the workgroup writes one row of sums to the
// workspace, and a second kernel adds these rows, all in a fixed order.

#include "zs_layer_device.h"

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

// The sum over a team's lanes, in every one of them.  Between waves it goes
// through part, two of which take turns, so that one barrier per sum will do:
// who writes part k again has passed the barrier of part k + 1, before which
// every wave has read part k.
template <int TEAM, int N>
__device__ __forceinline__ void team_sums(float (&x)[N], float (*part)[N][16], int& turn) {
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = wave_sum(x[k]);
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

template <int DT, int TEAM, int E, int WG, bool LAYER>
__global__ __launch_bounds__(WG) void norm_kernel(NormArgs a) {
  constexpr int V = kPack<DT>, J = E / V, TEAMS = WG / TEAM;
  __shared__ float part[2][1][16];
  int turn = 0;
  const int lane = threadIdx.x % TEAM;
  const int team = __builtin_amdgcn_readfirstlane(threadIdx.x / TEAM);
  Vals<V> gamma[J], beta[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = (lane + j * TEAM) * V;
    gamma[j] = ld_weights<V>(a.gamma, a.wdt, c, a.cols - c, 1.0f);
    beta[j] = ld_weights<V>(a.beta, a.wdt, c, a.cols - c, 0.0f);
  }
  const float n = static_cast<float>(a.cols);
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * TEAMS; r0 < a.rows;
       r0 += static_cast<int64_t>(gridDim.x) * TEAMS) {
    const int64_t r = r0 + team;
    if (TEAMS > 1 && r >= a.rows) return;  // a team of one wave waits for nobody
    const char* x = reinterpret_cast<const char*>(a.x.at + r * a.x.pitch);
    float t[J][V];
    Pack<DT> q[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = (lane + j * TEAM) * V;
      q[j] = ld_some<DT>(x + c * kSize<DT>, a.cols - c);
    }
    if (a.residual.at) {
      const char* res = reinterpret_cast<const char*>(a.residual.at + r * a.residual.pitch);
      char* total = reinterpret_cast<char*>(a.total.at + r * a.total.pitch);
      Pack<DT> p[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int c = (lane + j * TEAM) * V;
        p[j] = ld_some<DT>(res + c * kSize<DT>, a.cols - c);
      }
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int c = (lane + j * TEAM) * V;
        float f[V];
        widen<DT>(q[j], t[j]);
        widen<DT>(p[j], f);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = t[j][i] + f[i];
        q[j] = narrow<DT>(f);
        st_some<DT>(total + c * kSize<DT>, a.cols - c, q[j]);
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
        if constexpr (LAYER) t[j][i] = i < left ? t[j][i] - mean : 0.0f;
        s[0] += t[j][i] * t[j][i];
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
      st_some<DT>(y + c * kSize<DT>, a.cols - c, narrow<DT>(f));
    }
    if (lane == 0) {
      if (LAYER && a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
}

struct NormGradArgs {
  Rows dy, x, dres, dx;
  const void* gamma;
  const float* mean;
  const float* rstd;
  float* partial;  // or null: no gradients of weights
  int64_t rows, beta_at;
  int cols, wdt;
};

template <int DT, int J>
struct GradRow {
  Pack<DT> dy[J], x[J];
  float mean, rstd;
};

template <int DT, int TEAM, int J, bool LAYER>
__device__ __forceinline__ GradRow<DT, J> ld_grad_row(const NormGradArgs& a, int64_t r, int lane) {
  GradRow<DT, J> g{};
  if (r >= a.rows) return g;
  const char* dy = reinterpret_cast<const char*>(a.dy.at + r * a.dy.pitch);
  const char* x = reinterpret_cast<const char*>(a.x.at + r * a.x.pitch);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = (lane + j * TEAM) * kPack<DT>;
    g.dy[j] = ld_some<DT>(dy + c * kSize<DT>, a.cols - c);
    g.x[j] = ld_some<DT>(x + c * kSize<DT>, a.cols - c);
  }
  if constexpr (LAYER) g.mean = a.mean[r];
  g.rstd = a.rstd[r];
  return g;
}

template <int DT, int TEAM, int E, int WG, bool LAYER, bool BETA>
__global__ __launch_bounds__(WG) void norm_grad_kernel(NormGradArgs a) {
  constexpr int V = kPack<DT>, J = E / V, TEAMS = WG / TEAM;
  __shared__ float part[2][LAYER ? 2 : 1][16];
  extern __shared__ float sums[];  // cols, where there are several teams
  int turn = 0;
  const int lane = threadIdx.x % TEAM;
  const int team = __builtin_amdgcn_readfirstlane(threadIdx.x / TEAM);
  Vals<V> gamma[J];
  float acc_g[J][V], acc_b[J][V];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = (lane + j * TEAM) * V;
    gamma[j] = ld_weights<V>(a.gamma, a.wdt, c, a.cols - c, 1.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) acc_g[j][i] = acc_b[j][i] = 0.0f;
  }
  const float n = static_cast<float>(a.cols);
  const int64_t step = static_cast<int64_t>(gridDim.x) * TEAMS;
  int64_t r = static_cast<int64_t>(blockIdx.x) * TEAMS + team;
  GradRow<DT, J> next = ld_grad_row<DT, TEAM, J, LAYER>(a, r, lane);
  // every team of the workgroup makes as many turns as its first
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * TEAMS; r0 < a.rows; r0 += step, r += step) {
    const GradRow<DT, J> g = next;
    next = ld_grad_row<DT, TEAM, J, LAYER>(a, r + step, lane);
    float h[J][V], t[J][V];
    float s[LAYER ? 2 : 1] = {};
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int left = a.cols - (lane + j * TEAM) * V;
      widen<DT>(g.x[j], h[j]);
      widen<DT>(g.dy[j], t[j]);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (LAYER) h[j][i] = h[j][i] - g.mean;
        h[j][i] = i < left ? h[j][i] * g.rstd : 0.0f;
        acc_g[j][i] += t[j][i] * h[j][i];
        if constexpr (BETA) acc_b[j][i] += t[j][i];
        t[j][i] = t[j][i] * gamma[j].v[i];
        s[0] += t[j][i] * h[j][i];
        if constexpr (LAYER) s[1] += t[j][i];
      }
    }
    team_sums<TEAM>(s, part, turn);
    const float c2 = s[0] / n, c1 = LAYER ? s[LAYER ? 1 : 0] / n : 0.0f;
    if (r >= a.rows) continue;
    char* dx = reinterpret_cast<char*>(a.dx.at + r * a.dx.pitch);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = (lane + j * TEAM) * V;
      float f[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float u = LAYER ? t[j][i] - c1 : t[j][i];
        f[i] = (u - h[j][i] * c2) * g.rstd;
      }
      if (a.dres.at) {
        const char* dres = reinterpret_cast<const char*>(a.dres.at + r * a.dres.pitch);
        float d[V];
        widen<DT>(ld_some<DT>(dres + c * kSize<DT>, a.cols - c), d);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = f[i] + d[i];
      }
      st_some<DT>(dx + c * kSize<DT>, a.cols - c, narrow<DT>(f));
    }
  }
  if (!a.partial) return;
  const auto out = [&](float(&acc)[J][V], float* to) {
    if constexpr (TEAMS == 1) {
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int c = (lane + j * TEAM) * V + i;
          if (c < a.cols) to[c] = acc[j][i];
        }
    } else {
      for (int k = 0; k < TEAMS; ++k) {
        __syncthreads();
        if (team != k) continue;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const int c = (lane + j * TEAM) * V + i;
            if (c < a.cols) sums[c] = k == 0 ? acc[j][i] : sums[c] + acc[j][i];
          }
      }
      __syncthreads();
      for (int c = threadIdx.x; c < a.cols; c += WG) to[c] = sums[c];
    }
  };
  float* to = a.partial + static_cast<int64_t>(blockIdx.x) * a.cols;
  out(acc_g, to);
  if constexpr (BETA) {
    if (TEAMS > 1) __syncthreads();
    out(acc_b, to + a.beta_at);
  }
}

// The rows of sums, added in their order: 32 columns and 32 parts of the rows
// per workgroup.
constexpr int kJoinCols = 32, kJoinParts = 32;

struct NormJoinArgs {
  const float* partial;
  int64_t beta_at;
  void* dgamma;
  void* dbeta;
  int parts, cols, dt, accumulate;
};

__global__ __launch_bounds__(kJoinCols* kJoinParts) void norm_join_kernel(NormJoinArgs a) {
  __shared__ float sums[kJoinParts][kJoinCols];
  const bool beta = blockIdx.y != 0;
  void* to = beta ? a.dbeta : a.dgamma;
  if (!to) return;
  const int k = threadIdx.x % kJoinCols, p = threadIdx.x / kJoinCols;
  const int c = blockIdx.x * kJoinCols + k;
  const float* from = a.partial + (beta ? a.beta_at : 0);
  float s = 0.0f;
  if (c < a.cols)
    for (int i = p; i < a.parts; i += kJoinParts) s += from[static_cast<int64_t>(i) * a.cols + c];
  sums[p][k] = s;
  __syncthreads();
  if (p != 0 || c >= a.cols) return;
#pragma unroll
  for (int i = 1; i < kJoinParts; ++i) s += sums[i][k];
  st_value(to, a.dt, c, a.accumulate ? ld_value(to, a.dt, c) + s : s);
}

// Calls f(dtype, team, elements per lane).
template <class F>
void with_shape(int dt, int cols, F&& f) {
  with_gdt(dt, [&](auto d) {
    if (cols <= 512) f(d, IC<64>{}, IC<8>{});
    else if (cols <= 1024) f(d, IC<64>{}, IC<16>{});
    else if (cols <= 2048) f(d, IC<128>{}, IC<16>{});
    else if (cols <= 4096) f(d, IC<256>{}, IC<16>{});
    else if (cols <= 8192) f(d, IC<512>{}, IC<16>{});
    else f(d, IC<1024>{}, IC<16>{});
  });
}
static_assert(ZS_NORM_MAX_COLS == 1024 * 16, "the longest row is a team of 1024 lanes");

constexpr int norm_group(int team) { return team == kWave ? 4 * kWave : team; }
constexpr int grad_group(int team) { return team > 512 ? team : 512; }

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
  with_shape(L.dt, L.cols, [&](auto d, auto team, auto e) {
    constexpr int TEAM = decltype(team)::value, WG = norm_group(TEAM), TEAMS = WG / TEAM;
    const int64_t groups = (L.rows + TEAMS - 1) / TEAMS;
    const int64_t most = static_cast<int64_t>(cu_count()) * (2048 / WG);
    const dim3 grid(static_cast<unsigned>(groups < most ? groups : most));
    if (L.layer)
      norm_kernel<decltype(d)::value, TEAM, decltype(e)::value, WG, true><<<grid, WG, 0, L.stream>>>(a);
    else
      norm_kernel<decltype(d)::value, TEAM, decltype(e)::value, WG, false><<<grid, WG, 0, L.stream>>>(a);
  });
  return hipGetLastError();
}

hipError_t launch_norm_grad(const NormGradLaunch& L) {
  const bool sums = L.dgamma || L.dbeta;
  NormGradArgs a;
  a.dy = L.dy;
  a.x = L.x;
  a.dres = L.dres;
  a.dx = L.dx;
  a.gamma = L.gamma;
  a.mean = L.mean;
  a.rstd = L.rstd;
  a.partial = sums ? L.partial : nullptr;
  a.rows = L.rows;
  a.beta_at = static_cast<int64_t>(kNormParts) * L.cols;
  a.cols = L.cols;
  a.wdt = L.wdt;
  int parts = 0;
  if (L.rows > 0) {
    with_shape(L.dt, L.cols, [&](auto d, auto team, auto e) {
      constexpr int TEAM = decltype(team)::value, WG = grad_group(TEAM), TEAMS = WG / TEAM;
      const int64_t groups = (L.rows + TEAMS - 1) / TEAMS;
      int64_t most = static_cast<int64_t>(cu_count()) * (1024 / WG);
      if (most > kNormParts) most = kNormParts;
      parts = static_cast<int>(groups < most ? groups : most);
      const size_t lds = TEAMS > 1 ? sizeof(float) * static_cast<size_t>(L.cols) : 0;
      const auto go = [&](auto layer, auto beta) {
        norm_grad_kernel<decltype(d)::value, TEAM, decltype(e)::value, WG, decltype(layer)::value != 0,
                         decltype(beta)::value != 0>
            <<<dim3(static_cast<unsigned>(parts)), WG, lds, L.stream>>>(a);
      };
      L.layer ? go(IC<1>{}, IC<1>{}) : L.dbeta ? go(IC<0>{}, IC<1>{}) : go(IC<0>{}, IC<0>{});
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!sums || (L.rows == 0 && L.accumulate)) return hipSuccess;
  NormJoinArgs j;
  j.partial = L.partial;
  j.beta_at = a.beta_at;
  j.dgamma = L.dgamma;
  j.dbeta = L.dbeta;
  j.parts = parts;
  j.cols = L.cols;
  j.dt = L.gdt;
  j.accumulate = L.accumulate ? 1 : 0;
  norm_join_kernel<<<dim3(static_cast<unsigned>((L.cols + kJoinCols - 1) / kJoinCols), L.dbeta ? 2 : 1),
                     kJoinCols * kJoinParts, 0, L.stream>>>(j);
  return hipGetLastError();
}

}  // namespace zs
