// zs_embed.hip -- lookup in an embedding table, and the table's gradient.
//
// The lookup copies rows: each lane takes 16 bytes of a token's row.  The
// gradient is a sum over the tokens that name a row, without atomics so that its
// order is fixed: the tokens are sorted by row (a stable radix sort, so that
// equal rows keep the tokens' order), the sorted list is cut into chunks, and a
// wave sums the rows of dy of one chunk and 1 KiB of columns.  A table's row
// whose tokens all lie in one chunk is written at once; the others' sums go to
// the workspace, and a last kernel adds them in their order.  The pass over dy
// and the table's gradient bounds it; with accumulate = 0 the table is cleared by
// the workgroups that the sort leaves free.

#include "zs_layer_device.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

constexpr int kEmbedLoads = 4;  // packs of a lane

// What the clearing workgroups hold per CU, and stores of a lane at a time.
constexpr int kClearLanes = 1024, kClearLoads = 4;
template <int WG>
constexpr int64_t kClearEach = int64_t{WG} * kClearLoads;

struct EmbedArgs {
  const void* ids;
  const char* table;
  const void* pos_ids;
  const char* pos_table;
  Rows y;
  int64_t tokens, rows, first_row, pos_rows;
  uint32_t cols, packs;  // packs: of a row
  float scale;
};

template <bool WIDE>
__device__ __forceinline__ int64_t ld_id(const void* ids, int64_t t) {
  return WIDE ? static_cast<const int64_t*>(ids)[t] : static_cast<const int32_t*>(ids)[t];
}
// The row of a table of `rows` rows from `first` on that an id names, or -1.
__device__ __forceinline__ int64_t row_of(int64_t id, int64_t first, int64_t rows) {
  return id >= first && id - first < rows ? id - first : -1;
}

template <int DT, int TDT, bool WIDE, bool POS>
__global__ __launch_bounds__(kBlock) void embed_kernel(EmbedArgs a) {
  constexpr int V = kPack<DT>;
  const int64_t all = a.tokens * a.packs;
  constexpr int kEach = kBlock * kEmbedLoads;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kEach; i0 < all;
       i0 += static_cast<int64_t>(gridDim.x) * kEach) {
    // the workgroup's first token and pack, then 32-bit steps from there
    const int64_t t0 = i0 / a.packs;
    const uint32_t k0 = static_cast<uint32_t>(i0 - t0 * a.packs);
    Vals<V> f[kEmbedLoads], g[kEmbedLoads];
    int64_t r[kEmbedLoads], p[kEmbedLoads];
#pragma unroll
    for (int u = 0; u < kEmbedLoads; ++u) {
      const int64_t t = t0 + (k0 + u * kBlock + threadIdx.x) / a.packs;
      r[u] = p[u] = -1;
      if (t < a.tokens) {
        r[u] = row_of(ld_id<WIDE>(a.ids, t), a.first_row, a.rows);
        if constexpr (POS) p[u] = row_of(ld_id<WIDE>(a.pos_ids, t), 0, a.pos_rows);
      }
    }
#pragma unroll
    for (int u = 0; u < kEmbedLoads; ++u) {
      const uint32_t c = ((k0 + u * kBlock + threadIdx.x) % a.packs) * V;
      const int n = static_cast<int>(a.cols - c);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        f[u].v[i] = 0.0f;
        g[u].v[i] = -0.0f;  // nothing is added
      }
      if (r[u] >= 0) f[u] = ld_vals<V, TDT>(a.table + (r[u] * a.cols + c) * kSize<TDT>, n, 0.0f);
      if constexpr (POS)
        if (p[u] >= 0) g[u] = ld_vals<V, TDT>(a.pos_table + (p[u] * a.cols + c) * kSize<TDT>, n, 0.0f);
    }
#pragma unroll
    for (int u = 0; u < kEmbedLoads; ++u) {
      const uint32_t k = k0 + u * kBlock + threadIdx.x;
      const int64_t t = t0 + k / a.packs;
      const uint32_t c = (k % a.packs) * V;
      if (t < a.tokens) {
        float y[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          y[i] = r[u] >= 0 ? f[u].v[i] * a.scale : 0.0f;
          if constexpr (POS) y[i] = y[i] + g[u].v[i];
        }
        st_some<DT>(reinterpret_cast<char*>(a.y.at + t * a.y.pitch) + c * kSize<DT>,
                    static_cast<int>(a.cols - c), narrow<DT>(y));
      }
    }
  }
}

// ---- the tokens in the order of their rows ------------------------------------

struct SortArgs {
  const void* ids;
  TokenRow* list;     // the outcome
  TokenRow* other;    // before or after a pass, where many workgroups sort
  uint32_t* counts;   // per tile and digit
  uint32_t* long_rows;  // set to 0
  int64_t rows, first_row;
  int32_t tokens, tile;  // tile: tokens of a workgroup
  int passes, bits;   // bits: of a digit
  char* clear;        // bytes that the other workgroups clear
  int64_t clear_bytes;
};

template <bool WIDE>
__device__ __forceinline__ uint32_t ld_row_of(const SortArgs& a, int t) {
  const int64_t r = row_of(ld_id<WIDE>(a.ids, t), a.first_row, a.rows);
  return static_cast<uint32_t>(r >= 0 ? r : a.rows);  // tokens without a row come last
}

// Zeros by workgroup i of n of WG lanes.
template <int WG>
__device__ __forceinline__ void clear_part(char* at, int64_t bytes, int64_t i, int64_t n) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(at), hi = lo + bytes;
  const uintptr_t mid = (lo + 15) & ~uintptr_t{15}, end = hi & ~uintptr_t{15};
  if (i == 0) {  // the ends, in 16-bit steps
    const uintptr_t head = mid < hi ? mid : hi;
    for (uintptr_t x = lo + 2 * threadIdx.x; x < head; x += 2 * WG) *reinterpret_cast<uint16_t*>(x) = 0;
    for (uintptr_t x = (end > head ? end : head) + 2 * threadIdx.x; x < hi; x += 2 * WG)
      *reinterpret_cast<uint16_t*>(x) = 0;
  }
  if (end <= mid) return;
  const int64_t units = static_cast<int64_t>((end - mid) / 16);
  u32x4a16* to = reinterpret_cast<u32x4a16*>(mid);
  const u32x4a16 zero{0, 0, 0, 0};
  int64_t u = i * kClearEach<WG> + threadIdx.x;
  for (; u - threadIdx.x + kClearEach<WG> <= units; u += n * kClearEach<WG>) {
#pragma unroll
    for (int k = 0; k < kClearLoads; ++k) __builtin_nontemporal_store(zero, to + u + k * WG);
  }
#pragma unroll
  for (int k = 0; k < kClearLoads; ++k)
    if (u + k * WG < units) __builtin_nontemporal_store(zero, to + u + k * WG);
}

// Lanes of the wave whose digit is this lane's, of those that are live.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, bool live, int bits) {
  uint64_t same = __ballot(live);
  for (int b = 0; b < bits; ++b) {
    const bool set = (digit >> b) & 1u;
    const uint64_t with = __ballot(set);
    same &= set ? with : ~with;
  }
  return same;
}

// The lane's place among the live lanes of its digit, counted on from at[digit],
// which moves on.  LDS operations of one wave are in order.
__device__ __forceinline__ uint32_t take_place(uint32_t* at, uint32_t digit, bool live, int bits,
                                               int lane) {
  const uint64_t same = same_digit(digit, live, bits);
  const uint64_t below = same & ((uint64_t{1} << lane) - 1);
  uint32_t place = 0;
  if (live) place = __hip_atomic_load(at + digit, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
  __builtin_amdgcn_wave_barrier();
  if (live && below == 0)
    __hip_atomic_store(at + digit, place + static_cast<uint32_t>(__popcll(same)), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_WORKGROUP);
  __builtin_amdgcn_wave_barrier();
  return place + static_cast<uint32_t>(__popcll(below));
}

// The exclusive sums, over the lanes of a workgroup, of one value each; *all: the
// sum of all.  work: a word per wave; every lane calls it.
template <int WG>
__device__ __forceinline__ uint32_t scan_lanes(uint32_t mine, uint32_t* work, uint32_t* all) {
  uint32_t x = mine;
#pragma unroll
  for (int s = 1; s < kWave; s *= 2) {
    const uint32_t y = __shfl_up(x, s, kWave);
    if (static_cast<int>(threadIdx.x % kWave) >= s) x += y;
  }
  if (threadIdx.x % kWave == kWave - 1) work[threadIdx.x / kWave] = x;
  __syncthreads();
  uint32_t before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < WG / kWave; ++w) {
    const uint32_t n = work[w];
    if (w < static_cast<int>(threadIdx.x / kWave)) before += n;
    sum += n;
  }
  __syncthreads();
  *all = sum;
  return before + x - mine;
}

// One workgroup sorts, the others clear.  Each wave holds a run of the tokens,
// K to a lane, and counts its digits; sums over digits and waves turn the counts
// into the places of each wave's tokens.  Between two passes only the tokens'
// numbers move, through LDS; their rows are read again.
constexpr int kSortLanes = 1024, kSortWaves = kSortLanes / kWave;

template <bool WIDE, int K>
__global__ __launch_bounds__(kSortLanes) void sort_alone_kernel(SortArgs a) {
  __shared__ uint32_t counts[kSortWaves << kSortBits];
  __shared__ uint32_t work[kSortWaves];
  __shared__ uint16_t order[kSortLanes * K];
  static_assert(kSortLanes * K <= 1 << 16, "a token's number in 16 bits");
  if (blockIdx.x != 0) {
    clear_part<kSortLanes>(a.clear, a.clear_bytes, blockIdx.x - 1, gridDim.x - 1);
    return;
  }
  if (threadIdx.x == 0) *a.long_rows = 0;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int t0 = wave * kWave * K + lane;
  const int digits = 1 << a.bits;
  uint32_t* mine = counts + wave * digits;
  uint32_t row[K], token[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    token[k] = t0 + k * kWave;
    row[k] = t0 + k * kWave < a.tokens ? ld_row_of<WIDE>(a, t0 + k * kWave) : 0;
  }
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
    for (int i = threadIdx.x; i < kSortWaves * digits; i += kSortLanes) counts[i] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (t0 + k * kWave < a.tokens) atomicAdd(mine + ((row[k] >> shift) & (digits - 1)), 1u);
    __syncthreads();
    const int d = threadIdx.x;
    uint32_t n[kSortWaves], sum = 0, all;
    if (d < digits) {
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        n[w] = counts[w * digits + d];
        sum += n[w];
      }
    }
    uint32_t at = scan_lanes<kSortLanes>(sum, work, &all);
    if (d < digits) {
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        counts[w * digits + d] = at;
        at += n[w];
      }
    }
    __syncthreads();
    const bool last = pass == a.passes - 1;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const bool live = t0 + k * kWave < a.tokens;
      const uint32_t place = take_place(mine, (row[k] >> shift) & (digits - 1), live, a.bits, lane);
      if (!live) continue;
      if (last)
        a.list[place] = TokenRow{row[k], token[k]};
      else
        order[place] = static_cast<uint16_t>(token[k]);
    }
    if (last) break;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (t0 + k * kWave < a.tokens) token[k] = order[t0 + k * kWave];
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (t0 + k * kWave < a.tokens) row[k] = ld_row_of<WIDE>(a, token[k]);
  }
}
static_assert(1 << kSortBits <= kSortLanes, "a digit per lane");
static_assert(kSortAlone <= 16 * kSortLanes, "16 tokens per lane");

// Many workgroups: each has a tile of the tokens, and each of its waves a run of
// the tile.  Two kernels per pass: one counts the tiles' digits, the other adds up
// the counts before its tile and digit and puts the tokens in their places.
constexpr int kTileWaves = kBlock / kWave;

// Calls f(step's first token, K tokens' rows and numbers, how many of the lane's
// are there) over a wave's run of the tile.
template <bool WIDE, bool FIRST, class F>
__device__ __forceinline__ void for_run(const SortArgs& a, const TokenRow* from, F&& f) {
  constexpr int K = 8;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int run = a.tile / kTileWaves;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tile + static_cast<int64_t>(wave) * run;
  const int64_t t1 = t0 + run < a.tokens ? t0 + run : a.tokens;
  for (int64_t t = t0; t < t1; t += K * kWave) {
    TokenRow q[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t x = t + k * kWave + lane;
      q[k] = TokenRow{0, 0};
      if (x < t1) {
        if constexpr (FIRST)
          q[k] = TokenRow{ld_row_of<WIDE>(a, static_cast<int>(x)), static_cast<uint32_t>(x)};
        else
          q[k] = from[x];
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) f(q[k], t + k * kWave + lane < t1);
  }
}

template <bool WIDE, bool FIRST>
__global__ __launch_bounds__(kBlock) void sort_count_kernel(SortArgs a, const TokenRow* from, int shift,
                                                           int tiles) {
  if (static_cast<int>(blockIdx.x) >= tiles) {
    clear_part<kBlock>(a.clear, a.clear_bytes, blockIdx.x - tiles, gridDim.x - tiles);
    return;
  }
  __shared__ uint32_t counts[1 << kSortBits];
  if (FIRST && blockIdx.x == 0 && threadIdx.x == 0) *a.long_rows = 0;
  const int digits = 1 << a.bits;
  for (int i = threadIdx.x; i < digits; i += kBlock) counts[i] = 0;
  __syncthreads();
  for_run<WIDE, FIRST>(a, from, [&](TokenRow q, bool live) {
    if (live) atomicAdd(counts + ((q.row >> shift) & (digits - 1)), 1u);
  });
  __syncthreads();
  for (int i = threadIdx.x; i < digits; i += kBlock) a.counts[(blockIdx.x << a.bits) + i] = counts[i];
}

template <bool WIDE, bool FIRST>
__global__ __launch_bounds__(kBlock) void sort_place_kernel(SortArgs a, const TokenRow* from, TokenRow* to,
                                                           int shift) {
  __shared__ uint32_t counts[kTileWaves << kSortBits];
  __shared__ uint32_t work[kTileWaves];
  const int digits = 1 << a.bits;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  uint32_t* mine = counts + wave * digits;
  for (int i = threadIdx.x; i < kTileWaves * digits; i += kBlock) counts[i] = 0;
  __syncthreads();
  for_run<WIDE, FIRST>(a, from, [&](TokenRow q, bool live) {
    if (live) atomicAdd(mine + ((q.row >> shift) & (digits - 1)), 1u);
  });
  __syncthreads();
  uint32_t carry = 0;
  for (int d0 = 0; d0 < digits; d0 += kBlock) {
    const int d = d0 + threadIdx.x;
    uint32_t sum = 0, before = 0, all;
    if (d < digits) {
      const uint32_t* at = a.counts + d;
      const int tiles = gridDim.x, own = blockIdx.x;
#pragma unroll 8
      for (int t = 0; t < tiles; ++t) {
        const uint32_t n = at[t << a.bits];
        sum += n;
        if (t < own) before += n;
      }
    }
    uint32_t place = carry + scan_lanes<kBlock>(sum, work, &all) + before;
    carry += all;
    if (d < digits)
      for (int w = 0; w < kTileWaves; ++w) {
        const uint32_t n = counts[w * digits + d];
        counts[w * digits + d] = place;
        place += n;
      }
  }
  __syncthreads();
  for_run<WIDE, FIRST>(a, from, [&](TokenRow q, bool live) {
    const uint32_t place = take_place(mine, (q.row >> shift) & (digits - 1), live, a.bits, lane);
    if (live) to[place] = q;
  });
}

// ---- the sums -------------------------------------------------------------------

struct SumArgs {
  const TokenRow* list;
  Rows dy;
  void* grad;
  float* partial;       // two rows of sums per window
  uint32_t* long_rows;  // how many, and the windows in which they begin
  int64_t rows;
  int32_t tokens, windows;
  int cols, slabs;      // slabs: of a wave's columns
  float scale;
};

constexpr int kSumLoads = 8;  // rows in flight per wave

// V columns of a row of the gradient, n of them there.
template <int V, int GDT, bool ADD>
__device__ __forceinline__ void st_grad(const SumArgs& a, int64_t row, int c, int n, const Vals<V>& sum) {
  if (n <= 0) return;
  char* to = static_cast<char*>(a.grad) + (row * a.cols + c) * kSize<GDT>;
  Vals<V> f;
  if constexpr (ADD) f = ld_vals<V, GDT>(to, n, 0.0f);
#pragma unroll
  for (int i = 0; i < V; ++i) f.v[i] = ADD ? f.v[i] + sum.v[i] * a.scale : sum.v[i] * a.scale;
  st_vals<V, GDT>(to, n, f);
}

// Calls f(unit) for each unit that is this wave's.
template <class F>
__device__ __forceinline__ void for_units(int64_t units, F&& f) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWaves +
                   __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
       i < units; i += static_cast<int64_t>(gridDim.x) * kWaves)
    f(i);
}

// A window is kWindow places of the sorted list.  The wave of a window and slab of
// columns sums every table row whose tokens begin in the window, as far as they go,
// if they are at most kWindow.  The tokens of a row that has more (a long row) are
// summed by each window that they meet: where they begin, to the window's second row
// of sums, elsewhere to its first; sum_join_kernel adds these.
//
// What is where shows in masks of the 3 * kWindow places from kWindow before the
// window's first: bit l of `on` says that place l holds the row of place l - 1.
constexpr int kWindow = 16;

struct Window {
  uint32_t row, token;  // of place `lane`
  uint64_t on, live;
};
__device__ __forceinline__ Window ld_window(const SumArgs& a, int64_t w, int lane) {
  const int64_t p = (w - 1) * kWindow + lane;
  const uint32_t none = static_cast<uint32_t>(a.rows);
  TokenRow q{none, 0};
  if (lane < 3 * kWindow && p >= 0 && p < a.tokens) q = a.list[p];
  const uint32_t before = __shfl_up(q.row, 1, kWave);
  Window x;
  x.row = q.row;
  x.token = q.token;
  x.live = __ballot(q.row != none);
  x.on = __ballot(lane > 0 && q.row == before) & x.live;
  return x;
}
// Whether the row that begins at place s has more than kWindow tokens.
__device__ __forceinline__ bool is_long(uint64_t on, int s) {
  constexpr uint64_t all = (uint64_t{1} << kWindow) - 1;
  return ((on >> (s + 1)) & all) == all;
}
// The last place up to l at which a row begins; 0: at none from 1 on.
__device__ __forceinline__ int begin_of(uint64_t on, int l) {
  const uint64_t begins = ~on & ((uint64_t{2} << l) - 2);
  return begins ? 63 - __builtin_clzll(begins) : 0;
}

template <int DT, int GDT, bool ADD>
__device__ __forceinline__ void sum_unit(const SumArgs& a, int64_t unit) {
  constexpr int V = kPack<DT>;
  const int lane = threadIdx.x % kWave;
  const int64_t w = unit / a.slabs;
  const int slab = static_cast<int>(unit - w * a.slabs);
  const int c = (slab * kWave + lane) * V, n = a.cols - c;
  const Window x = ld_window(a, w, lane);
  const uint64_t stop = ~x.on;
  int l = kWindow;
  bool head = false;  // a long row that began before the window
  if (x.on >> l & 1) {
    const int s = begin_of(x.on, l);
    head = s == 0 || is_long(x.on, s);
    if (!head) l += __builtin_ctzll(stop >> l);  // its own window's
  }
  int end = 2 * kWindow;
  bool tail = false;
  if (x.on >> end & 1) {
    const int s = begin_of(x.on, end);
    if (s >= kWindow) {  // or it is the head, which meets all of the window
      tail = is_long(x.on, s);
      if (!tail) end += __builtin_ctzll(stop >> end);
    }
  }
  const int live = 64 - __builtin_clzll(x.live | 1);
  end = end < live ? end : live;
  if (tail && slab == 0 && lane == 0) {
    const uint32_t at = __hip_atomic_fetch_add(a.long_rows, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    a.long_rows[1 + at] = static_cast<uint32_t>(w);
  }
  Vals<V> sum;
#pragma unroll
  for (int i = 0; i < V; ++i) sum.v[i] = 0.0f;
  for (; l < end; l += kSumLoads) {
    Pack<DT> p[kSumLoads];
#pragma unroll
    for (int u = 0; u < kSumLoads; ++u) {
      if (l + u >= end) break;
      const uint32_t t = __builtin_amdgcn_readlane(x.token, l + u);
      p[u] = ld_some<DT>(reinterpret_cast<const char*>(a.dy.at + t * a.dy.pitch) +
                             static_cast<int64_t>(c) * kSize<DT>,
                         n);
    }
#pragma unroll
    for (int u = 0; u < kSumLoads; ++u) {
      if (l + u >= end) break;
      float f[V];
      widen<DT>(p[u], f);
#pragma unroll
      for (int i = 0; i < V; ++i) sum.v[i] = sum.v[i] + f[i];
      const bool last = l + u + 1 == end;
      if (!last && (x.on >> (l + u + 1) & 1)) continue;
      const bool part = head || (last && tail);
      if (part) {
        float* to = a.partial + (2 * w + (head ? 0 : 1)) * a.cols + c;
        st_vals<V, kF32>(reinterpret_cast<char*>(to), n, sum);
      } else {
        st_grad<V, GDT, ADD>(a, __builtin_amdgcn_readlane(x.row, l + u), c, n, sum);
      }
      head = false;
#pragma unroll
      for (int i = 0; i < V; ++i) sum.v[i] = 0.0f;
    }
  }
}

template <int DT, int GDT, bool ADD>
__global__ __launch_bounds__(kBlock) void sum_kernel(SumArgs a) {
  for_units(static_cast<int64_t>(a.windows) * a.slabs,
            [&](int64_t unit) { sum_unit<DT, GDT, ADD>(a, unit); });
}

// A long row's sum: a workgroup per row and 256 columns, whose waves take equal
// shares of its windows' sums.
constexpr int kJoinV = 4, kJoinSlab = kWave * kJoinV, kJoinLoads = 8;

template <int GDT, bool ADD>
__global__ __launch_bounds__(kBlock) void sum_join_kernel(SumArgs a) {
  __shared__ Vals<kJoinV> sums[kWaves][kWave];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t units = static_cast<int64_t>(a.long_rows[0]) * a.slabs;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int64_t k = unit / a.slabs, w = a.long_rows[1 + k];
    const int c = (static_cast<int>(unit - k * a.slabs) * kWave + lane) * kJoinV, n = a.cols - c;
    const uint32_t row = a.list[(w + 1) * kWindow].row;
    int64_t more = 1;  // windows after w that it meets
    while (true) {
      const int64_t x = (w + 1 + more + lane) * kWindow;
      const uint64_t stops = ~__ballot(x < a.tokens && a.list[x < a.tokens ? x : 0].row == row);
      if (stops != 0) {
        more += __builtin_ctzll(stops);
        break;
      }
      more += kWave;
    }
    // rows of sums 2 w + 1, 2 (w + 1), 2 (w + 2) ...
    const int64_t each = (more + kWaves) / kWaves;
    const int64_t i1 = (wave + 1) * each < more + 1 ? (wave + 1) * each : more + 1;
    Vals<kJoinV> sum;
#pragma unroll
    for (int i = 0; i < kJoinV; ++i) sum.v[i] = 0.0f;
    for (int64_t i = wave * each; i < i1; i += kJoinLoads) {
      Vals<kJoinV> f[kJoinLoads];
#pragma unroll
      for (int u = 0; u < kJoinLoads; ++u) {
#pragma unroll
        for (int q = 0; q < kJoinV; ++q) f[u].v[q] = 0.0f;
        const int64_t at = i + u == 0 ? 2 * w + 1 : 2 * (w + i + u);
        if (i + u < i1 && n > 0)
          f[u] = ld_vals<kJoinV, kF32>(reinterpret_cast<const char*>(a.partial + at * a.cols + c), n, 0.0f);
      }
#pragma unroll
      for (int u = 0; u < kJoinLoads; ++u)
#pragma unroll
        for (int q = 0; q < kJoinV; ++q) sum.v[q] = sum.v[q] + f[u].v[q];
    }
    sums[wave][lane] = sum;
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int i = 1; i < kWaves; ++i)
#pragma unroll
        for (int q = 0; q < kJoinV; ++q) sum.v[q] = sum.v[q] + sums[i][lane].v[q];
      st_grad<kJoinV, GDT, ADD>(a, row, c, n, sum);
    }
    __syncthreads();
  }
}

int bits_of(uint64_t x) { return x == 0 ? 1 : 64 - __builtin_clzll(x); }

size_t up256(size_t x) { return (x + 255u) & ~static_cast<size_t>(255u); }

// Tokens per tile: no more tiles than kTilesMost, so that each may add up the
// counts of all.
constexpr int kTilesMost = 256, kTileStep = 2048;
int64_t tile_of(int64_t tokens) {
  const int64_t steps = (tokens + kTileStep - 1) / kTileStep;
  return (steps + kTilesMost - 1) / kTilesMost * kTileStep;
}

}  // namespace

EmbedLayout embed_layout(int64_t tokens, int64_t cols) {
  EmbedLayout l;
  const bool alone = tokens <= kSortAlone;
  const size_t list = up256(sizeof(TokenRow) * static_cast<size_t>(tokens));
  const size_t windows = static_cast<size_t>((tokens + kWindow - 1) / kWindow);
  const size_t tiles = alone ? 0 : static_cast<size_t>((tokens + tile_of(tokens) - 1) / tile_of(tokens));
  l.list = 0;
  l.other = list;
  l.counts = l.other + (alone ? 0 : list);
  l.long_rows = l.counts + (sizeof(uint32_t) << kSortBits) * tiles;
  l.partial = l.long_rows + up256(sizeof(uint32_t) * (windows + 1));
  l.total = l.partial + up256(sizeof(float) * 2 * windows * static_cast<size_t>(cols));
  return l;
}

hipError_t launch_embed(const EmbedLaunch& L) {
  EmbedArgs a;
  a.ids = L.ids;
  a.table = static_cast<const char*>(L.table);
  a.pos_ids = L.pos_ids;
  a.pos_table = static_cast<const char*>(L.pos_table);
  a.y = L.y;
  a.tokens = L.tokens;
  a.rows = L.rows;
  a.first_row = L.first_row;
  a.pos_rows = L.pos_rows;
  a.cols = static_cast<uint32_t>(L.cols);
  a.scale = L.scale;
  with_gdt(L.dt, [&](auto d) {
    constexpr int DT = decltype(d)::value;
    a.packs = (a.cols + kPack<DT> - 1) / kPack<DT>;
    const int64_t each = kBlock * kEmbedLoads;
    const int64_t groups = (L.tokens * a.packs + each - 1) / each;
    const dim3 grid(static_cast<unsigned>(groups < kMaxGroups ? groups : kMaxGroups));
    with_gdt(L.tdt, [&](auto t) {
      constexpr int TDT = decltype(t)::value;
      const auto go = [&](auto wide, auto pos) {
        embed_kernel<DT, TDT, decltype(wide)::value != 0, decltype(pos)::value != 0>
            <<<grid, kBlock, 0, L.stream>>>(a);
      };
      const auto pick = [&](auto wide) { L.pos_table ? go(wide, IC<1>{}) : go(wide, IC<0>{}); };
      L.wide_ids ? pick(IC<1>{}) : pick(IC<0>{});
    });
  });
  return hipGetLastError();
}

namespace {

hipError_t launch_sort(const EmbedGradLaunch& L, const EmbedLayout& lay) {
  SortArgs a;
  a.ids = L.ids;
  a.list = reinterpret_cast<TokenRow*>(L.workspace + lay.list);
  a.other = reinterpret_cast<TokenRow*>(L.workspace + lay.other);
  a.counts = reinterpret_cast<uint32_t*>(L.workspace + lay.counts);
  a.long_rows = reinterpret_cast<uint32_t*>(L.workspace + lay.long_rows);
  a.rows = L.rows;
  a.first_row = L.first_row;
  a.tokens = static_cast<int32_t>(L.tokens);
  a.tile = 0;
  const int key_bits = bits_of(static_cast<uint64_t>(L.rows));  // a row, or rows itself
  a.passes = (key_bits + kSortBits - 1) / kSortBits;
  a.bits = (key_bits + a.passes - 1) / a.passes;
  a.clear = static_cast<char*>(L.grad);
  a.clear_bytes = L.rows * L.cols * (L.gdt == kF32 ? 4 : 2);
  const bool alone = L.tokens <= kSortAlone;
  const int lanes = alone ? kSortLanes : kBlock;
  int64_t clearers = 0;
  if (!L.accumulate) {
    const int64_t most = int64_t{cu_count()} * (kClearLanes / lanes);
    clearers = a.clear_bytes / (16 * kClearLoads * lanes) + 1;
    if (clearers > most) clearers = most;
  }
  if (alone) {
    const dim3 grid(static_cast<unsigned>(1 + clearers));
    const auto go = [&](auto k) {
      if (L.wide_ids) sort_alone_kernel<true, decltype(k)::value><<<grid, kSortLanes, 0, L.stream>>>(a);
      else sort_alone_kernel<false, decltype(k)::value><<<grid, kSortLanes, 0, L.stream>>>(a);
    };
    if (L.tokens <= 1 * kSortLanes) go(IC<1>{});
    else if (L.tokens <= 4 * kSortLanes) go(IC<4>{});
    else if (L.tokens <= 8 * kSortLanes) go(IC<8>{});
    else go(IC<16>{});
    return hipGetLastError();
  }
  a.tile = static_cast<int32_t>(tile_of(L.tokens));
  const int tiles = static_cast<int>((L.tokens + a.tile - 1) / a.tile);
  const TokenRow* from = nullptr;
  TokenRow* to = a.passes % 2 ? a.list : a.other;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
    const dim3 grid(static_cast<unsigned>(tiles)), first(static_cast<unsigned>(tiles + clearers));
    if (pass > 0) {
      sort_count_kernel<false, false><<<grid, kBlock, 0, L.stream>>>(a, from, shift, tiles);
      sort_place_kernel<false, false><<<grid, kBlock, 0, L.stream>>>(a, from, to, shift);
    } else if (L.wide_ids) {
      sort_count_kernel<true, true><<<first, kBlock, 0, L.stream>>>(a, from, shift, tiles);
      sort_place_kernel<true, true><<<grid, kBlock, 0, L.stream>>>(a, from, to, shift);
    } else {
      sort_count_kernel<false, true><<<first, kBlock, 0, L.stream>>>(a, from, shift, tiles);
      sort_place_kernel<false, true><<<grid, kBlock, 0, L.stream>>>(a, from, to, shift);
    }
    from = to;
    to = to == a.list ? a.other : a.list;
  }
  return hipGetLastError();
}

__global__ __launch_bounds__(kSortLanes) void clear_kernel(char* at, int64_t bytes) {
  clear_part<kSortLanes>(at, bytes, blockIdx.x, gridDim.x);
}

}  // namespace

hipError_t launch_embed_grad(const EmbedGradLaunch& L) {
  if (L.tokens == 0) {
    clear_kernel<<<dim3(static_cast<unsigned>(cu_count())), kSortLanes, 0, L.stream>>>(
        static_cast<char*>(L.grad), L.rows * L.cols * (L.gdt == kF32 ? 4 : 2));
    return hipGetLastError();
  }
  const EmbedLayout lay = embed_layout(L.tokens, L.cols);
  const hipError_t e = launch_sort(L, lay);
  if (e != hipSuccess) return e;
  SumArgs a;
  a.list = reinterpret_cast<const TokenRow*>(L.workspace + lay.list);
  a.dy = L.dy;
  a.grad = L.grad;
  a.partial = reinterpret_cast<float*>(L.workspace + lay.partial);
  a.long_rows = reinterpret_cast<uint32_t*>(L.workspace + lay.long_rows);
  a.rows = L.rows;
  a.tokens = static_cast<int32_t>(L.tokens);
  a.windows = static_cast<int32_t>((L.tokens + kWindow - 1) / kWindow);
  a.cols = L.cols;
  a.scale = L.scale;
  with_gdt(L.gdt, [&](auto g) {
    constexpr int GDT = decltype(g)::value;
    const auto go = [&](auto add) {
      constexpr bool ADD = decltype(add)::value != 0;
      with_gdt(L.dt, [&](auto d) {
        constexpr int DT = decltype(d)::value, kSlab = kWave * kPack<DT>;
        a.slabs = (L.cols + kSlab - 1) / kSlab;
        const int64_t groups = (static_cast<int64_t>(a.windows) * a.slabs + kWaves - 1) / kWaves;
        sum_kernel<DT, GDT, ADD><<<dim3(static_cast<unsigned>(groups < kMaxGroups ? groups : kMaxGroups)), kBlock,
                                   0, L.stream>>>(a);
      });
      if (L.tokens <= kWindow) return;  // no long row
      a.slabs = (L.cols + kJoinSlab - 1) / kJoinSlab;
      const int64_t most = int64_t{cu_count()} * 8;
      const int64_t units = L.tokens / (kWindow + 1) * a.slabs;
      sum_join_kernel<GDT, ADD><<<dim3(static_cast<unsigned>(units < most ? units : most)), kBlock, 0, L.stream>>>(a);
    };
    L.accumulate ? go(IC<1>{}) : go(IC<0>{});
  });
  return hipGetLastError();
}

}  // namespace zs
