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

template <int DT, int TEAM, int J, bool WHOLE, bool STREAM>
__device__ __forceinline__ void ld_row(const Rows& rows, int64_t r, int lane, int cols, Pack<DT> (&q)[J]) {
  const char* at = reinterpret_cast<const char*>(rows.at + r * rows.pitch);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = (lane + j * TEAM) * kPack<DT>;
    q[j] = ld_some<DT, WHOLE, STREAM>(at + c * kSize<DT>, cols - c);
  }
}

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

template <int DT, int TEAM, int E, int WG, bool LAYER, bool WHOLE, bool STREAM>
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
    float t[J][V];
    Pack<DT> q[J];
    ld_row<DT, TEAM, J, WHOLE, STREAM>(a.x, r, lane, a.cols, q);
    if (a.residual.at) {
      char* total = reinterpret_cast<char*>(a.total.at + r * a.total.pitch);
      Pack<DT> p[J];
      ld_row<DT, TEAM, J, WHOLE, STREAM>(a.residual, r, lane, a.cols, p);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int c = (lane + j * TEAM) * V;
        float f[V];
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

struct NormGradArgs {
  Rows dy, x, dres, dx;
  const void* gamma;
  const float* mean;
  const float* rstd;
  float* partial;  // or null: no sums over rows here
  void* dgamma;    // of the workgroups from `groups` on
  void* dbeta;
  int64_t rows, beta_at;
  int cols, wdt, groups, gdt, accumulate;
};

template <int DT, int J>
struct GradRow {
  Pack<DT> dy[J], x[J];
  float mean, rstd;
};

template <int DT, int TEAM, int J, bool LAYER, bool WHOLE>
__device__ __forceinline__ GradRow<DT, J> ld_grad_row(const NormGradArgs& a, int64_t r, int lane) {
  GradRow<DT, J> g{};
  if (r >= a.rows) return g;
  const char* dy = reinterpret_cast<const char*>(a.dy.at + r * a.dy.pitch);
  const char* x = reinterpret_cast<const char*>(a.x.at + r * a.x.pitch);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = (lane + j * TEAM) * kPack<DT>;
    g.dy[j] = ld_some<DT, WHOLE>(dy + c * kSize<DT>, a.cols - c);
    g.x[j] = ld_some<DT, WHOLE>(x + c * kSize<DT>, a.cols - c);
  }
  if constexpr (LAYER) g.mean = a.mean[r];
  g.rstd = a.rstd[r];
  return g;
}

// Makes the compiler forget what it computed of a pack.
template <int DT>
__device__ __forceinline__ void forget(Pack<DT>& q) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    auto x = q.x[i];
    asm volatile("" : "+v"(x));
    q.x[i] = x;
  }
}

// h = (x - mean) * rstd of a pack, zeros where the row has ended within it.  Packs
// wholly beyond the row (WHOLE) give values that only products with their dy, which
// is 0, see.
template <int DT, bool LAYER, bool WHOLE>
__device__ __forceinline__ void normed(const Pack<DT>& x, float mean, float rstd, int left,
                                       float (&h)[kPack<DT>]) {
  widen<DT>(x, h);
#pragma unroll
  for (int i = 0; i < kPack<DT>; ++i) {
    if constexpr (LAYER) h[i] = h[i] - mean;
    h[i] = WHOLE || i < left ? h[i] * rstd : 0.0f;
  }
}

// The weights' gradients of 8 packs of columns, straight from all rows: each 8 lanes
// of the workgroup take a row at a time.
constexpr int kColumnLanes = 8;

template <int DT, int WG, bool LAYER, bool BETA, bool WHOLE>
__device__ __forceinline__ void column_sums(const NormGradArgs& a, int slab) {
  constexpr int V = kPack<DT>, kLoads = 4, kRows = WG / kColumnLanes;
  __shared__ float sums[2][WG / kWave][kColumnLanes * V];
  const int lane = threadIdx.x % kColumnLanes;
  const int c = (slab * kColumnLanes + lane) * V, n = a.cols - c;
  float acc_g[V], acc_b[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc_g[i] = acc_b[i] = 0.0f;
  for (int64_t r = threadIdx.x / kColumnLanes; r < a.rows; r += kRows * kLoads) {
    Pack<DT> dy[kLoads], x[kLoads];
    float mean[kLoads], rstd[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int64_t q = r + u * kRows;
      const int there = q < a.rows ? n : 0;
      dy[u] = ld_some<DT, WHOLE, false>(reinterpret_cast<const char*>(a.dy.at + q * a.dy.pitch) + c * kSize<DT>, there);
      x[u] = ld_some<DT, WHOLE, false>(reinterpret_cast<const char*>(a.x.at + q * a.x.pitch) + c * kSize<DT>, there);
      mean[u] = LAYER && there > 0 ? a.mean[q] : 0.0f;
      rstd[u] = there > 0 ? a.rstd[q] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      float h[V], t[V];
      normed<DT, LAYER, WHOLE>(x[u], mean[u], rstd[u], r + u * kRows < a.rows ? n : 0, h);
      widen<DT>(dy[u], t);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        acc_g[i] = __builtin_fmaf(t[i], h[i], acc_g[i]);
        if constexpr (BETA) acc_b[i] += t[i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int s = kColumnLanes; s < kWave; s *= 2) {
      acc_g[i] += __shfl_xor(acc_g[i], s, kWave);
      if constexpr (BETA) acc_b[i] += __shfl_xor(acc_b[i], s, kWave);
    }
  if (threadIdx.x % kWave < kColumnLanes) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      sums[0][threadIdx.x / kWave][lane * V + i] = acc_g[i];
      if constexpr (BETA) sums[1][threadIdx.x / kWave][lane * V + i] = acc_b[i];
    }
  }
  __syncthreads();
  const int which = threadIdx.x / (kColumnLanes * V), k = threadIdx.x % (kColumnLanes * V);
  const int64_t col = static_cast<int64_t>(slab) * kColumnLanes * V + k;
  void* to = which == 0 ? a.dgamma : a.dbeta;
  if (which > BETA || !to || col >= a.cols) return;
  float s = sums[which][0][k];
#pragma unroll
  for (int w = 1; w < WG / kWave; ++w) s += sums[which][w][k];
  st_value(to, a.gdt, col, a.accumulate ? ld_value(to, a.gdt, col) + s : s);
}

// A lane's sums go to place (j * V + i) * TEAM + lane of a row of sums, so that
// all accesses of LDS and of the workspace are of neighbouring lanes; the join
// puts them in the order of the columns.
template <int DT, int TEAM, int E, int WG, bool LAYER, bool BETA, bool WHOLE>
__global__ __launch_bounds__(WG) void norm_grad_kernel(NormGradArgs a) {
  constexpr int V = kPack<DT>, J = E / V, TEAMS = WG / TEAM;
  if (static_cast<int>(blockIdx.x) >= a.groups) {
    column_sums<DT, WG, LAYER, BETA, WHOLE>(a, static_cast<int>(blockIdx.x) - a.groups);
    return;
  }
  __shared__ float part[2][LAYER ? 2 : 1][16];
  extern __shared__ float sums[];  // WG * E, where there are several teams
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
  const int64_t step = static_cast<int64_t>(a.groups) * TEAMS;
  int64_t r = static_cast<int64_t>(blockIdx.x) * TEAMS + team;
  // every team of the workgroup makes as many turns as its first
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * TEAMS; r0 < a.rows; r0 += step, r += step) {
    GradRow<DT, J> g = ld_grad_row<DT, TEAM, J, LAYER, WHOLE>(a, r, lane);
    Pack<DT> dres[J];
    if (a.dres.at && r < a.rows) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int c = (lane + j * TEAM) * V;
        dres[j] = ld_some<DT, WHOLE>(reinterpret_cast<const char*>(a.dres.at + r * a.dres.pitch) + c * kSize<DT>,
                              a.cols - c);
      }
    }
    float s[LAYER ? 2 : 1] = {};
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float h[V], t[V];
      normed<DT, LAYER, WHOLE>(g.x[j], g.mean, g.rstd, a.cols - (lane + j * TEAM) * V, h);
      widen<DT>(g.dy[j], t);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        acc_g[j][i] = __builtin_fmaf(t[i], h[i], acc_g[j][i]);
        if constexpr (BETA) acc_b[j][i] += t[i];
        t[i] = t[i] * gamma[j].v[i];
        s[0] = __builtin_fmaf(t[i], h[i], s[0]);
        if constexpr (LAYER) s[1] += t[i];
      }
    }
    team_sums<TEAM>(s, part, turn);
    const float c2 = s[0] / n, c1 = LAYER ? s[LAYER ? 1 : 0] / n : 0.0f;
    if (r >= a.rows) continue;
    char* dx = reinterpret_cast<char*>(a.dx.at + r * a.dx.pitch);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      // h and dy * gamma once more; of 16 elements they are computed again, since to
      // keep them would take registers that 16 waves per CU do not have
      const int c = (lane + j * TEAM) * V;
      float h[V], t[V];
      if constexpr (E > 8) {
        forget(g.x[j]);
        forget(g.dy[j]);
      }
      normed<DT, LAYER, WHOLE>(g.x[j], g.mean, g.rstd, a.cols - c, h);
      widen<DT>(g.dy[j], t);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        t[i] = t[i] * gamma[j].v[i];
        if constexpr (LAYER) t[i] = t[i] - c1;
        t[i] = (t[i] - h[i] * c2) * g.rstd;
      }
      if (a.dres.at) {
        widen<DT>(dres[j], h);
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] = t[i] + h[i];
      }
      st_some<DT, WHOLE>(dx + c * kSize<DT>, a.cols - c, narrow<DT>(t));
    }
  }
  if (!a.partial) return;
  const auto out = [&](float(&acc)[J][V], float* to) {
    if constexpr (TEAMS == 1) {
#pragma unroll
      for (int k = 0; k < E; ++k) to[k * TEAM + lane] = acc[k / V][k % V];
    } else {
#pragma unroll
      for (int k = 0; k < E; ++k) sums[(team * E + k) * TEAM + lane] = acc[k / V][k % V];
      __syncthreads();
      for (int c = threadIdx.x; c < E * TEAM; c += WG) {
        float s = sums[c];
#pragma unroll
        for (int k = 1; k < TEAMS; ++k) s += sums[k * E * TEAM + c];
        to[c] = s;
      }
    }
  };
  float* to = a.partial + static_cast<int64_t>(blockIdx.x) * (E * TEAM);
  out(acc_g, to);
  if constexpr (BETA) {
    if (TEAMS > 1) __syncthreads();
    out(acc_b, to + a.beta_at);
  }
}

// The rows of sums, added in a fixed order: 16 places and 64 parts of the rows
// per workgroup, eight loads of a lane in flight.
constexpr int kJoinCols = 16, kJoinParts = 64, kJoinLoads = kNormParts / kJoinParts;

struct NormJoinArgs {
  const float* partial;
  int64_t beta_at;
  void* dgamma;
  void* dbeta;
  int parts, width, team, pack, cols, dt, accumulate;  // width: of a row of sums
};

__global__ __launch_bounds__(kJoinCols* kJoinParts) void norm_join_kernel(NormJoinArgs a) {
  __shared__ float sums[kJoinParts][kJoinCols];
  const bool beta = blockIdx.y != 0;
  void* to = beta ? a.dbeta : a.dgamma;
  if (!to) return;
  const int k = threadIdx.x % kJoinCols, p = threadIdx.x / kJoinCols;
  const int at = blockIdx.x * kJoinCols + k;  // width is a multiple of kJoinCols
  const int own = at / a.team, c = (at % a.team + own / a.pack * a.team) * a.pack + own % a.pack;
  const float* from = a.partial + (beta ? a.beta_at : 0) + at;
  float x[kJoinLoads];
#pragma unroll
  for (int i = 0; i < kJoinLoads; ++i) {
    const int row = p + i * kJoinParts;
    x[i] = row < a.parts && c < a.cols ? from[static_cast<int64_t>(row) * a.width] : 0.0f;
  }
  float s = x[0];
#pragma unroll
  for (int i = 1; i < kJoinLoads; ++i) s += x[i];
  sums[p][k] = s;
#pragma unroll
  for (int d = kJoinParts / 2; d > 0; d /= 2) {
    __syncthreads();
    if (p < d) sums[p][k] = s = s + sums[p + d][k];
  }
  if (p != 0 || c >= a.cols) return;
  st_value(to, a.dt, c, a.accumulate ? ld_value(to, a.dt, c) + s : s);
}

// Calls f(dtype, team, elements per lane) for the smallest team that holds a row.
// A lane of the backward pass holds 8 elements (16 of the longest rows), so that
// its sums leave registers for 16 waves per CU.  The forward pass takes 16, half
// the waves per row (16384 x 4096 bf16, layer norm 47.8 us; 63.9 with 8).
template <int E, class F>
void with_shape(int dt, int cols, F&& f) {
  with_gdt(dt, [&](auto d) {
    if (cols <= 64 * 8) f(d, IC<64>{}, IC<8>{});
    else if (cols <= 64 * E) f(d, IC<64>{}, IC<E>{});
    else if (cols <= 128 * E) f(d, IC<128>{}, IC<E>{});
    else if (cols <= 256 * E) f(d, IC<256>{}, IC<E>{});
    else if (cols <= 512 * E) f(d, IC<512>{}, IC<E>{});
    else if (cols <= 1024 * E) f(d, IC<1024>{}, IC<E>{});
    else f(d, IC<1024>{}, IC<16>{});
  });
}
static_assert(ZS_NORM_MAX_COLS == 1024 * 16, "the longest row is a team of 1024 lanes");

// Workgroups of the forward pass: with a residual one row per team, which ends
// (16384 x 4096 bf16 85.9 us, 6.2 TB/s; 92.9 with 1024 lanes per CU that go on to
// further rows); without one, and for rows of 1024 lanes, as many elements per CU
// at a time (16384 x 4096 bf16, layer norm 47.8 us, one row per team 52.0; 4096 x
// 16384 56.9 and 70.9).
constexpr int kNormHeld = 16384;
// Where a call reads and writes more than this, its rows do not stay in the 256 MB
// cache from one kernel of a model to the next, and it reads past that (16384 x 4096 with a
// residual 85.9 us, 89.8 read through it); smaller ones may have been left there
// by the kernel before (32768 x 1024 bf16 22.4 us, read past it 27.4).
constexpr int64_t kNormCached = int64_t{192} << 20;

// The weights' gradients of few rows come from workgroups of the same launch that
// read these rows again (8 lanes to a row, 64 or 128 rows at a time), not from rows
// of sums and a second launch.  us in one launch / in two, layer norm, bf16: 333 x
// 1001 7.2 / 9.1, 64 x 768 6.1 / 9.0, 1024 x 768 7.8 / 9.3, 2048 x 768 16.5 / 10.0,
// 512 x 4096 8.3 / 14.5, 1024 x 4096 15.4 / 16.8, 256 x 16384 15.1 / 27.5.
constexpr int64_t kNormFewRows = 1024, kNormFewElems = int64_t{1} << 22;

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
  const bool stream = L.rows * L.cols * (L.dt == kF32 ? 4 : 2) * (L.residual.at ? 4 : 2) > kNormCached;
  with_shape<16>(L.dt, L.cols, [&](auto d, auto team, auto e) {
    constexpr int TEAM = decltype(team)::value, WG = norm_group(TEAM), TEAMS = WG / TEAM;
    const int64_t groups = (L.rows + TEAMS - 1) / TEAMS;
    const int64_t most = L.residual.at && TEAM < 1024 ? kMaxGroups / (WG > kBlock ? WG / kBlock : 1)
                                                     : int64_t{cu_count()} * (kNormHeld / decltype(e)::value / WG);
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
  // in place the rows' workgroups write what the columns' would read
  const bool few = sums && L.rows <= kNormFewRows && L.rows * L.cols <= kNormFewElems &&
                   L.dx.at != L.dy.at && L.dx.at != L.x.at;
  a.partial = sums && !few ? L.partial : nullptr;
  a.dgamma = L.dgamma;
  a.dbeta = L.dbeta;
  a.gdt = L.gdt;
  a.accumulate = L.accumulate ? 1 : 0;
  a.rows = L.rows;
  a.cols = L.cols;
  a.wdt = L.wdt;
  NormJoinArgs j;
  j.parts = 0;
  {
    with_shape<8>(L.dt, L.cols, [&](auto d, auto team, auto e) {
      constexpr int TEAM = decltype(team)::value, WG = grad_group(TEAM), TEAMS = WG / TEAM;
      const int64_t groups = (L.rows + TEAMS - 1) / TEAMS;
      int64_t most = static_cast<int64_t>(cu_count()) * (1024 / WG);
      if (most > kNormParts) most = kNormParts;
      j.parts = static_cast<int>(groups < most ? groups : most);
      j.team = TEAM;
      j.pack = kPack<decltype(d)::value>;
      j.width = decltype(e)::value * TEAM;
      a.beta_at = j.beta_at = static_cast<int64_t>(kNormParts) * j.width;
      if (j.parts == 0) return;
      a.groups = j.parts;
      constexpr int kSlab = kColumnLanes * kPack<decltype(d)::value>;
      const int columns = few ? (L.cols + kSlab - 1) / kSlab : 0;
      const dim3 grid(static_cast<unsigned>(a.groups + columns));
      const size_t lds = TEAMS > 1 ? sizeof(float) * decltype(e)::value * WG : 0;
      const auto go = [&](auto layer, auto beta, auto whole) {
        norm_grad_kernel<decltype(d)::value, TEAM, decltype(e)::value, WG, decltype(layer)::value != 0,
                         decltype(beta)::value != 0, decltype(whole)::value != 0>
            <<<grid, WG, lds, L.stream>>>(a);
      };
      const auto pick = [&](auto whole) {
        L.layer ? go(IC<1>{}, IC<1>{}, whole) : L.dbeta ? go(IC<0>{}, IC<1>{}, whole) : go(IC<0>{}, IC<0>{}, whole);
      };
      L.cols % kPack<decltype(d)::value> == 0 ? pick(IC<1>{}) : pick(IC<0>{});
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!sums || few) return hipSuccess;
  j.partial = L.partial;
  j.dgamma = L.dgamma;
  j.dbeta = L.dbeta;
  j.cols = L.cols;
  j.dt = L.gdt;
  j.accumulate = L.accumulate ? 1 : 0;
  norm_join_kernel<<<dim3(static_cast<unsigned>(j.width / kJoinCols), L.dbeta ? 2 : 1),
                     kJoinCols * kJoinParts, 0, L.stream>>>(j);
  return hipGetLastError();
}

}  // namespace zs
