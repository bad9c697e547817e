// zs_norm_grad.hip -- the norms' backward pass.
//
// A row stays in its team's registers as in the forward pass (zs_norm.hip), whose
// mean and root it is given.
//
// The weights' gradients are sums over rows.  Each lane keeps those of its own
// columns in registers over all rows that its team takes; the teams of a workgroup
// add theirs in LDS, the workgroup writes one row of sums to the workspace, and a
// second kernel adds these rows, all in a fixed order.  Two workgroups of 8 waves per
// CU, without the next row in flight: 16384 x 4096 bf16 with a gradient that passes
// by 93.5 us in all, three 102 to 107, four 107.5, one with the next row 116, two
// with it 94.5; 8192 x 768 16.0, 15.0, 18.8, 19.7 and 16.6.
//
// dy, x and dres are read past the cache whatever their size (us so and through it,
// bf16: 16384 x 4096 with a gradient that passes by 93.4 / 100.2, 32768 x 4096 151 /
// 153, 65536 x 1024 75.5 / 77.7, 32768 x 1024 42.4 / 43.2).  Inputs of less than 100
// MB, which the kernel before may have left there, pay for it: 8192 x 768 15.0 / 13.5,
// 16384 x 768 22.2 / 20.0, 4096 x 4096 30.9 / 27.5.

#include "zs_norm_device.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

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
    g.dy[j] = ld_some<DT, WHOLE>(dy, c, a.cols);
    g.x[j] = ld_some<DT, WHOLE>(x, c, a.cols);
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

// h = (x - mean) * rstd of a pack, zeros where the row has ended within it.  Of packs
// wholly beyond the row (WHOLE) it is -mean * rstd, which may be infinite: a row's sums
// leave it out.
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
      const int there = q < a.rows ? a.cols : 0;  // columns of the row
      const char* at_dy = reinterpret_cast<const char*>(a.dy.at + q * a.dy.pitch);
      const char* at_x = reinterpret_cast<const char*>(a.x.at + q * a.x.pitch);
      dy[u] = ld_some<DT, WHOLE, false>(at_dy, c, there);
      x[u] = ld_some<DT, WHOLE, false>(at_x, c, there);
      mean[u] = LAYER && there > 0 ? a.mean[q] : 0.0f;
      rstd[u] = there > 0 ? a.rstd[q] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      float h[V], t[V];
      settle<DT, WHOLE>(dy[u], c, a.cols);
      settle<DT, WHOLE>(x[u], c, a.cols);
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
  const int team = team_of<TEAM>();
  Vals<V> gamma[J];
  float acc_g[J][V], acc_b[J][V];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = (lane + j * TEAM) * V;
    gamma[j] = ld_weights<V>(a.gamma, a.wdt, c, a.cols, 1.0f);
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
      const char* at = reinterpret_cast<const char*>(a.dres.at + r * a.dres.pitch);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int c = (lane + j * TEAM) * V;
        dres[j] = ld_some<DT, WHOLE>(at, c, a.cols);
      }
    }
    float s[LAYER ? 2 : 1] = {};
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = (lane + j * TEAM) * V;
      float h[V], t[V];
      settle<DT, WHOLE>(g.dy[j], c, a.cols);
      settle<DT, WHOLE>(g.x[j], c, a.cols);
      normed<DT, LAYER, WHOLE>(g.x[j], g.mean, g.rstd, a.cols - c, h);
      widen<DT>(g.dy[j], t);
      const float before = s[0];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        acc_g[j][i] = __builtin_fmaf(t[i], h[i], acc_g[j][i]);
        if constexpr (BETA) acc_b[j][i] += t[i];
        t[i] = t[i] * gamma[j].v[i];
        s[0] = __builtin_fmaf(t[i], h[i], s[0]);
        if constexpr (LAYER) s[1] += t[i];
      }
      // beyond the row t is 0, but 0 * h need not be
      if (WHOLE && c >= a.cols) s[0] = before;
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
        settle<DT, WHOLE>(dres[j], c, a.cols);
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
// per workgroup, eight loads of a lane in flight.  16 places are half of a line of the
// cache, so two workgroups read each (16384 x 4096: 16.1 MiB of 8).
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

// The weights' gradients of few rows come from workgroups of the same launch that
// read these rows again (8 lanes to a row, 64 or 128 rows at a time), not from rows
// of sums and a second launch.  us in one launch / in two, layer norm, bf16: 333 x
// 1001 7.2 / 9.1, 64 x 768 6.1 / 9.0, 1024 x 768 7.8 / 9.3, 2048 x 768 16.5 / 10.0,
// 512 x 4096 8.3 / 14.5, 1024 x 4096 15.4 / 16.8, 256 x 16384 15.1 / 27.5.
constexpr int64_t kNormFewRows = 1024, kNormFewElems = int64_t{1} << 22;

constexpr int grad_group(int team) { return team > 512 ? team : 512; }

}  // namespace

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
        L.layer   ? go(IC<1>{}, IC<1>{}, whole)
        : L.dbeta ? go(IC<0>{}, IC<1>{}, whole)
                  : go(IC<0>{}, IC<0>{}, whole);
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
