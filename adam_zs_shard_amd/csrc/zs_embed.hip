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
  TokenRow* a;       // the list, which ends up in a
  TokenRow* b;
  uint32_t* counts;  // per digit and tile
  int64_t rows, first_row;
  int32_t tokens, tiles;
  int passes, bits;  // of a digit
  char* clear;       // or null: bytes that the other workgroups clear
  int64_t clear_bytes;
};

template <bool WIDE>
__device__ __forceinline__ TokenRow ld_token(const SortArgs& a, int t) {
  const int64_t r = row_of(ld_id<WIDE>(a.ids, t), a.first_row, a.rows);
  return TokenRow{static_cast<uint32_t>(r >= 0 ? r : a.rows), static_cast<uint32_t>(t)};
}

// Zeros by workgroups i of n of WG lanes.
template <int WG>
__device__ __forceinline__ void clear_bytes(char* at, int64_t bytes, int64_t i, int64_t n) {
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
  for (int64_t u = i * WG + threadIdx.x; u < units; u += n * WG)
    __builtin_nontemporal_store(u32x4a16{0, 0, 0, 0}, reinterpret_cast<u32x4a16*>(mid) + u);
}

// Lanes of the wave whose digit is this lane's, of those that are live.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, bool live, int bits) {
  uint64_t same = __ballot(live);
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot(live && ((digit >> b) & 1u));
    same &= (digit >> b) & 1u ? set : ~set;
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

// Exclusive sums over the digits, in order of digit and then of part, of
// counts[part][digit] in LDS.  Every lane of a workgroup of WG calls it.
template <int WG>
__device__ __forceinline__ void scan_digits(uint32_t* counts, int parts, int digits, uint32_t* work) {
  uint32_t carry = 0;
  for (int d0 = 0; d0 < digits; d0 += WG) {
    const int d = d0 + threadIdx.x;
    uint32_t mine = 0;
    if (d < digits)
      for (int p = 0; p < parts; ++p) mine += counts[p * digits + d];
    // over the lanes
    uint32_t x = mine;
    for (int s = 1; s < kWave; s *= 2) {
      const uint32_t y = __shfl_up(x, s, kWave);
      if (static_cast<int>(threadIdx.x % kWave) >= s) x += y;
    }
    if (threadIdx.x % kWave == kWave - 1) work[threadIdx.x / kWave] = x;
    __syncthreads();
    uint32_t before = carry, all = carry;
    for (int w = 0; w < WG / kWave; ++w) {
      if (w < static_cast<int>(threadIdx.x / kWave)) before += work[w];
      all += work[w];
    }
    carry = all;
    uint32_t at = before + x - mine;
    if (d < digits)
      for (int p = 0; p < parts; ++p) {
        const uint32_t n = counts[p * digits + d];
        counts[p * digits + d] = at;
        at += n;
      }
    __syncthreads();
  }
}

// One workgroup sorts, the others clear.  Each of its waves has a run of the
// tokens and, per pass, a count of each digit in it; the sums over the digits
// turn the counts into the places where each wave's tokens go.
constexpr int kSortLanes = 1024, kSortWaves = kSortLanes / kWave;

template <bool WIDE>
__global__ __launch_bounds__(kSortLanes) void sort_alone_kernel(SortArgs a) {
  if (blockIdx.x != 0 || a.tokens == 0) {
    if (a.clear)
      clear_bytes<kSortLanes>(a.clear, a.clear_bytes, a.tokens == 0 ? blockIdx.x : blockIdx.x - 1,
                              a.tokens == 0 ? gridDim.x : gridDim.x - 1);
    return;
  }
  __shared__ uint32_t counts[kSortWaves << kSortBits];
  __shared__ uint32_t work[kSortWaves];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int each = (a.tokens + kSortLanes - 1) / kSortLanes * kWave;  // tokens per wave
  const int t0 = wave * each, t1 = t0 + each < a.tokens ? t0 + each : a.tokens;
  const int digits = 1 << a.bits;
  uint32_t* mine = counts + wave * digits;
  TokenRow* from = a.passes % 2 ? a.b : a.a;
  TokenRow* to = a.passes % 2 ? a.a : a.b;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
    for (int i = threadIdx.x; i < kSortWaves * digits; i += kSortLanes) counts[i] = 0;
    __syncthreads();
    for (int t = t0 + lane; t < t1; t += kWave) {
      const TokenRow q = pass == 0 ? ld_token<WIDE>(a, t) : from[t];
      atomicAdd(mine + ((q.row >> shift) & (digits - 1)), 1u);
    }
    __syncthreads();
    scan_digits<kSortLanes>(counts, kSortWaves, digits, work);
    for (int t = t0; t < t1; t += kWave) {
      const bool live = t + lane < t1;
      TokenRow q{0, 0};
      if (live) q = pass == 0 ? ld_token<WIDE>(a, t + lane) : from[t + lane];
      const uint32_t place = take_place(mine, (q.row >> shift) & (digits - 1), live, a.bits, lane);
      if (live) to[place] = q;
    }
    __syncthreads();
    TokenRow* x = from;
    from = to;
    to = x;
  }
}

// Tiles of kSortTile tokens, one workgroup each; three kernels per pass.
constexpr int kTileWaves = kBlock / kWave;

template <bool WIDE, bool FIRST>
__global__ __launch_bounds__(kBlock) void sort_count_kernel(SortArgs a, const TokenRow* from, int shift) {
  if (static_cast<int>(blockIdx.x) >= a.tiles) {
    clear_bytes<kBlock>(a.clear, a.clear_bytes, blockIdx.x - a.tiles, gridDim.x - a.tiles);
    return;
  }
  __shared__ uint32_t counts[1 << kSortBits];
  const int digits = 1 << a.bits;
  for (int i = threadIdx.x; i < digits; i += kBlock) counts[i] = 0;
  __syncthreads();
  const int t0 = blockIdx.x * kSortTile;
  const int t1 = t0 + kSortTile < a.tokens ? t0 + kSortTile : a.tokens;
  for (int t = t0 + threadIdx.x; t < t1; t += kBlock) {
    const TokenRow q = FIRST ? ld_token<WIDE>(a, t) : from[t];
    atomicAdd(counts + ((q.row >> shift) & (digits - 1)), 1u);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < digits; i += kBlock)
    a.counts[static_cast<int64_t>(i) * a.tiles + blockIdx.x] = counts[i];
}

// Exclusive sums over n counts, in place, by one workgroup.
__global__ __launch_bounds__(kSortLanes) void sort_scan_kernel(uint32_t* counts, int64_t n) {
  __shared__ uint32_t work[kSortWaves];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  uint32_t carry = 0;
  for (int64_t i0 = 0; i0 < n; i0 += 4 * kSortLanes) {
    const int64_t i = i0 + 4 * threadIdx.x;
    uint32_t c[4], mine = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[j] = i + j < n ? counts[i + j] : 0u;
      mine += c[j];
    }
    uint32_t x = mine;
    for (int s = 1; s < kWave; s *= 2) {
      const uint32_t y = __shfl_up(x, s, kWave);
      if (lane >= s) x += y;
    }
    if (lane == kWave - 1) work[wave] = x;
    __syncthreads();
    uint32_t before = carry, all = carry;
    for (int w = 0; w < kSortWaves; ++w) {
      if (w < wave) before += work[w];
      all += work[w];
    }
    carry = all;
    uint32_t at = before + x - mine;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (i + j < n) counts[i + j] = at;
      at += c[j];
    }
    __syncthreads();
  }
}

template <bool WIDE, bool FIRST>
__global__ __launch_bounds__(kBlock) void sort_place_kernel(SortArgs a, const TokenRow* from, TokenRow* to,
                                                           int shift) {
  __shared__ uint32_t counts[kTileWaves << kSortBits];
  const int digits = 1 << a.bits;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  constexpr int kEach = kSortTile / kTileWaves;
  uint32_t* mine = counts + wave * digits;
  for (int i = threadIdx.x; i < kTileWaves * digits; i += kBlock) counts[i] = 0;
  __syncthreads();
  const int t0 = blockIdx.x * kSortTile + wave * kEach;
  const int t1 = t0 + kEach < a.tokens ? t0 + kEach : a.tokens;
  for (int t = t0 + lane; t < t1; t += kWave) {
    const TokenRow q = FIRST ? ld_token<WIDE>(a, t) : from[t];
    atomicAdd(mine + ((q.row >> shift) & (digits - 1)), 1u);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < digits; i += kBlock) {
    uint32_t at = a.counts[static_cast<int64_t>(i) * a.tiles + blockIdx.x];
    for (int w = 0; w < kTileWaves; ++w) {
      const uint32_t n = counts[w * digits + i];
      counts[w * digits + i] = at;
      at += n;
    }
  }
  __syncthreads();
  for (int t = t0; t < t1; t += kWave) {
    const bool live = t + lane < t1;
    TokenRow q{0, 0};
    if (live) q = FIRST ? ld_token<WIDE>(a, t + lane) : from[t + lane];
    const uint32_t place = take_place(mine, (q.row >> shift) & (digits - 1), live, a.bits, lane);
    if (live) to[place] = q;
  }
}

// ---- the sums -------------------------------------------------------------------

struct SumArgs {
  const TokenRow* list;
  Rows dy;
  void* grad;
  float* partial;  // two rows of sums per chunk
  int64_t rows, chunks;
  int32_t tokens, chunk;
  int cols, slabs;  // slabs: of 64 packs of columns
  float scale;
};

constexpr int kSumLoads = 8;  // rows of dy in flight per wave

template <int DT, int GDT, bool ADD>
__device__ __forceinline__ void st_grad(const SumArgs& a, int64_t row, int c, int n,
                                        const float (&sum)[kPack<DT>]) {
  constexpr int V = kPack<DT>;
  if (n <= 0) return;
  const int64_t at = row * a.cols + c;
  char* to = static_cast<char*>(a.grad) + at * kSize<GDT>;
  float f[V];
  if constexpr (ADD) {
    const Vals<V> old = ld_vals<V, GDT>(to, n, 0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = old.v[i] + sum[i] * a.scale;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = sum[i] * a.scale;
  }
  if constexpr (V == kPack<GDT>) {
    st_some<GDT>(to, n, narrow<GDT>(f));
  } else if constexpr (V == 8) {  // fp32 gradient of 16-bit rows: two packs
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float g[4] = {f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]};
      st_some<kF32>(to + 16 * k, n - 4 * k, narrow<kF32>(g));
    }
  } else {  // 16-bit gradient of fp32 rows: half a pack
    const u32x2 q{narrow_pair<GDT>(f[0], f[1]), narrow_pair<GDT>(f[2], f[3])};
    if (n >= 4)
      *reinterpret_cast<u32x2*>(to) = q;
    else
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) reinterpret_cast<uint16_t*>(to)[i] = static_cast<uint16_t>(q[i / 2] >> (16 * (i % 2)));
  }
}

// Calls f(unit) for each unit that is this wave's.
template <class F>
__device__ __forceinline__ void for_units(int64_t units, F&& f) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWaves +
                   __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
       i < units; i += static_cast<int64_t>(gridDim.x) * kWaves)
    f(i);
}

// One wave per unit, a chunk and a slab.
template <int DT, int GDT, bool ADD>
__device__ __forceinline__ void sum_unit(const SumArgs& a, int64_t unit) {
  constexpr int V = kPack<DT>;
  const int lane = threadIdx.x % kWave;
  const int64_t chunk = unit / a.slabs;
  const int c = static_cast<int>(unit - chunk * a.slabs) * kWave * V + lane * V;
  const int n = a.cols - c;
  const uint32_t none = static_cast<uint32_t>(a.rows);
  const int t0 = static_cast<int>(chunk) * a.chunk;
  const int count = a.tokens - t0 < a.chunk ? a.tokens - t0 : a.chunk;
  TokenRow q{none, 0};
  if (lane < count) q = a.list[t0 + lane];
  const uint32_t before = t0 > 0 ? a.list[t0 - 1].row : none;
  const uint32_t after = t0 + count < a.tokens ? a.list[t0 + count].row : none;
  const int live = __popcll(__ballot(q.row != none));  // the tokens without a row come last
  float sum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) sum[i] = 0.0f;
  bool open = before != none && live > 0 &&
              before == static_cast<uint32_t>(__builtin_amdgcn_readlane(q.row, 0));
  for (int k = 0; k < live; k += kSumLoads) {
    Pack<DT> p[kSumLoads];
#pragma unroll
    for (int u = 0; u < kSumLoads; ++u) {
      if (k + u >= live) break;
      const uint32_t t = __builtin_amdgcn_readlane(q.token, k + u);
      p[u] = ld_some<DT>(reinterpret_cast<const char*>(a.dy.at + t * a.dy.pitch) +
                             static_cast<int64_t>(c) * kSize<DT>,
                         n);
    }
#pragma unroll
    for (int u = 0; u < kSumLoads; ++u) {
      if (k + u >= live) break;
      float f[V];
      widen<DT>(p[u], f);
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] = sum[i] + f[i];
      const uint32_t row = __builtin_amdgcn_readlane(q.row, k + u);
      const bool last = k + u + 1 == count;
      const uint32_t next =
          last ? after : static_cast<uint32_t>(__builtin_amdgcn_readlane(q.row, (k + u + 1) % kWave));
      const bool goes_on = last && next == row;
      if (next == row && !goes_on) continue;
      if (open || goes_on) {  // part of a row's sum: the chunk's first row, or its last
        float* to = a.partial + (2 * chunk + (open ? 0 : 1)) * a.cols + c;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i < n) to[i] = sum[i];
      } else {
        st_grad<DT, GDT, ADD>(a, row, c, n, sum);
      }
      open = false;
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] = 0.0f;
    }
  }
}

template <int DT, int GDT, bool ADD>
__global__ __launch_bounds__(kBlock) void sum_kernel(SumArgs a) {
  for_units(a.chunks * a.slabs, [&](int64_t unit) { sum_unit<DT, GDT, ADD>(a, unit); });
}

// Adds the parts of the rows that begin in a chunk and go on in the next: one
// wave per chunk, but the last, and slab.
template <int DT, int GDT, bool ADD>
__device__ __forceinline__ void join_unit(const SumArgs& a, int64_t unit) {
  constexpr int V = kPack<DT>;
  const int lane = threadIdx.x % kWave;
  const int64_t chunk = unit / a.slabs;
  const int c = static_cast<int>(unit - chunk * a.slabs) * kWave * V + lane * V;
  const int n = a.cols - c;
  const uint32_t none = static_cast<uint32_t>(a.rows);
  const int64_t t0 = chunk * a.chunk;
  const uint32_t row = a.list[t0 + a.chunk - 1].row;
  if (row == none || a.list[t0 + a.chunk].row != row) return;
  if (t0 > 0 && a.list[t0 - 1].row == row) return;  // it began in an earlier chunk
  // a chunk whose first row it is: the chunk's first row of sums
  int64_t more = 1;
  while (true) {
    const int64_t x = chunk + more + lane;  // does the row go on behind chunk x?
    const bool on = x < a.chunks - 1 && a.list[(x + 1) * a.chunk].row == row;
    const uint64_t stops = ~__ballot(on);
    if (stops != 0) {
      more += __builtin_ctzll(stops);
      break;
    }
    more += kWave;
  }
  float sum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) sum[i] = 0.0f;
  const auto add = [&](int64_t at) {
    const float* from = a.partial + at * a.cols + c;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) sum[i] = sum[i] + from[i];
  };
  add(2 * chunk + 1);
  for (int64_t k = 1; k <= more; ++k) add(2 * (chunk + k));
  st_grad<DT, GDT, ADD>(a, row, c, n, sum);
}

template <int DT, int GDT, bool ADD>
__global__ __launch_bounds__(kBlock) void sum_join_kernel(SumArgs a) {
  for_units((a.chunks - 1) * a.slabs, [&](int64_t unit) { join_unit<DT, GDT, ADD>(a, unit); });
}

int bits_of(uint64_t x) { return x == 0 ? 1 : 64 - __builtin_clzll(x); }

size_t up256(size_t x) { return (x + 255u) & ~static_cast<size_t>(255u); }

}  // namespace

int embed_chunk(int64_t, int64_t) { return 32; }

EmbedLayout embed_layout(int64_t tokens, int64_t rows, int64_t cols) {
  EmbedLayout l;
  const size_t list = up256(sizeof(TokenRow) * static_cast<size_t>(tokens));
  const int chunk = embed_chunk(tokens, cols);
  const int64_t tiles = tokens > kSortAlone ? (tokens + kSortTile - 1) / kSortTile : 0;
  const int64_t chunks = (tokens + chunk - 1) / chunk;
  l.a = 0;
  l.b = list;
  l.counts = 2 * list;
  l.partial = l.counts + up256((sizeof(uint32_t) << kSortBits) * static_cast<size_t>(tiles));
  l.total = l.partial + up256(sizeof(float) * 2 * static_cast<size_t>(chunks) * static_cast<size_t>(cols));
  if (l.total == 0) l.total = 256;
  (void)rows;
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

hipError_t launch_sort(const EmbedGradLaunch& L, const EmbedLayout& lay, const TokenRow** list) {
  SortArgs a;
  a.ids = L.ids;
  a.a = reinterpret_cast<TokenRow*>(L.workspace + lay.a);
  a.b = reinterpret_cast<TokenRow*>(L.workspace + lay.b);
  a.counts = reinterpret_cast<uint32_t*>(L.workspace + lay.counts);
  a.rows = L.rows;
  a.first_row = L.first_row;
  a.tokens = static_cast<int32_t>(L.tokens);
  const int key_bits = bits_of(static_cast<uint64_t>(L.rows));  // rows stands for none
  a.passes = (key_bits + kSortBits - 1) / kSortBits;
  a.bits = (key_bits + a.passes - 1) / a.passes;
  a.clear = L.accumulate ? nullptr : static_cast<char*>(L.grad);
  const int size = L.gdt == kF32 ? 4 : 2;
  a.clear_bytes = L.rows * L.cols * size;
  *list = a.a;
  const bool alone = L.tokens <= kSortAlone;
  const int lanes = alone ? kSortLanes : kBlock;
  int64_t clearers = L.accumulate ? 0 : (a.clear_bytes / 16 + 4 * lanes - 1) / (4 * lanes) + 1;
  const int64_t most = static_cast<int64_t>(cu_count()) * (2048 / lanes);
  if (clearers > most) clearers = most;
  if (alone) {
    a.tiles = 0;
    const int64_t grid = clearers + (L.tokens > 0 ? 1 : 0);
    if (grid == 0) return hipSuccess;
    const dim3 g(static_cast<unsigned>(grid));
    if (L.wide_ids) sort_alone_kernel<true><<<g, kSortLanes, 0, L.stream>>>(a);
    else sort_alone_kernel<false><<<g, kSortLanes, 0, L.stream>>>(a);
    return hipGetLastError();
  }
  a.tiles = static_cast<int32_t>((L.tokens + kSortTile - 1) / kSortTile);
  const TokenRow* from = nullptr;
  TokenRow* to = a.passes % 2 ? a.a : a.b;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
    const dim3 tiles(static_cast<unsigned>(a.tiles));
    const dim3 first(static_cast<unsigned>(a.tiles + clearers));
    if (pass > 0) sort_count_kernel<false, false><<<tiles, kBlock, 0, L.stream>>>(a, from, shift);
    else if (L.wide_ids) sort_count_kernel<true, true><<<first, kBlock, 0, L.stream>>>(a, from, shift);
    else sort_count_kernel<false, true><<<first, kBlock, 0, L.stream>>>(a, from, shift);
    sort_scan_kernel<<<1, kSortLanes, 0, L.stream>>>(a.counts, static_cast<int64_t>(a.tiles) << a.bits);
    if (pass > 0) sort_place_kernel<false, false><<<tiles, kBlock, 0, L.stream>>>(a, from, to, shift);
    else if (L.wide_ids) sort_place_kernel<true, true><<<tiles, kBlock, 0, L.stream>>>(a, from, to, shift);
    else sort_place_kernel<false, true><<<tiles, kBlock, 0, L.stream>>>(a, from, to, shift);
    from = to;
    to = to == a.a ? a.b : a.a;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embed_grad(const EmbedGradLaunch& L) {
  const EmbedLayout lay = embed_layout(L.tokens, L.rows, L.cols);
  const TokenRow* list;
  const hipError_t e = launch_sort(L, lay, &list);
  if (e != hipSuccess || L.tokens == 0) return e;
  SumArgs a;
  a.list = list;
  a.dy = L.dy;
  a.grad = L.grad;
  a.partial = reinterpret_cast<float*>(L.workspace + lay.partial);
  a.rows = L.rows;
  a.tokens = static_cast<int32_t>(L.tokens);
  a.chunk = embed_chunk(L.tokens, L.cols);
  a.chunks = (L.tokens + a.chunk - 1) / a.chunk;
  a.cols = L.cols;
  a.scale = L.scale;
  with_gdt(L.dt, [&](auto d) {
    constexpr int DT = decltype(d)::value, kSlab = kWave * kPack<DT>;
    a.slabs = (L.cols + kSlab - 1) / kSlab;
    const int64_t groups = (a.chunks * a.slabs + kWaves - 1) / kWaves;
    const dim3 grid(static_cast<unsigned>(groups < kMaxGroups ? groups : kMaxGroups));
    with_gdt(L.gdt, [&](auto g) {
      constexpr int GDT = decltype(g)::value;
      const auto go = [&](auto add) {
        constexpr bool ADD = decltype(add)::value != 0;
        sum_kernel<DT, GDT, ADD><<<grid, kBlock, 0, L.stream>>>(a);
        if (a.chunks > 1) sum_join_kernel<DT, GDT, ADD><<<grid, kBlock, 0, L.stream>>>(a);
      };
      L.accumulate ? go(IC<1>{}) : go(IC<0>{});
    });
  });
  return hipGetLastError();
}

}  // namespace zs
