// zs_embed.hip -- lookup in an embedding table, and the table's gradient.
//
// The lookup copies rows, a lane 16 bytes of a token's.  HBM bounds it where the
// tokens are many (16384 of 4096 bf16 columns 34 us, 5.4 TB/s), latency where they
// are few: each row's address waits for the token's id.
//
// The gradient's row r is the sum of the rows of dy whose tokens name r, in the
// tokens' order and without atomics on floating-point numbers, so that it has the same
// bits every time.  The tokens are sorted by row, stably (one launch, or two per digit
// of the row for many tokens); the sorted list is cut into windows, and a wave sums
// the rows of dy of one window and 1 KiB of columns.  A table row with more tokens
// than a window has places is summed in parts, which go to the workspace, and a last
// kernel adds them in their order.  With accumulate = 0 the table is cleared by the launch that
// sorts, beside it; so the rows that tokens name are written twice, 45 MB of the 1.1
// GB that 16384 tokens of a 128256 x 4096 table move, for 20 us of sorting that
// nothing waits for.
//
// HBM bounds large tables and many tokens: 16384 tokens, 128256 x 4096 bf16: 165 us
// of clearing at 6.4 TB/s, 42 of sums at 4.7, 6 of parts.  131072 tokens added to
// 16032 x 1024 fp32: 23 us of sorting, 66 of sums at 5.4 TB/s, 17 of parts.  Few
// tokens wait: 500 added to 50257 x 768 4.4, 6 and 3.5 us for a MB or two.

#include "zs_layer_device.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

struct EmbedArgs {
  const void* ids;
  const char* table;
  const void* pos_ids;
  const char* pos_table;
  Rows y;
  int64_t tokens, rows, first_row, pos_rows;
  uint32_t cols, packs;  // packs: of a row
  uint32_t inverse;      // 2^32 / packs, rounded up
  float scale;
};

// k / packs for k < packs + kBlock: exact, since the product of the rounding of
// `inverse` (less than 1) and k stays below 2^32 / packs.
__device__ __forceinline__ uint32_t row_step(const EmbedArgs& a, uint32_t k) {
  if (a.packs >= kBlock) return k >= a.packs;
  return a.packs == 1 ? k : __umulhi(k, a.inverse);
}

template <bool WIDE>
__device__ __forceinline__ int64_t ld_id(const void* ids, int64_t t) {
  return WIDE ? static_cast<const int64_t*>(ids)[t] : static_cast<const int32_t*>(ids)[t];
}
// The row of a table of `rows` rows from `first` on that an id names, or -1.
__device__ __forceinline__ int64_t row_of(int64_t id, int64_t first, int64_t rows) {
  return id >= first && id - first < rows ? id - first : -1;
}

// A lane takes one pack and ends: 8192 tokens of 768 bf16 with positions 5.7 us, 5.9
// with two packs in flight, 7.4 with four; 16384 of 4096 34 us with one or two.
// WHOLE: rows of whole packs (the first 6.2 us without it).
template <int DT, int TDT, bool WIDE, bool POS, bool WHOLE>
__global__ __launch_bounds__(kBlock) void embed_kernel(EmbedArgs a) {
  constexpr int V = kPack<DT>;
  const int64_t all = a.tokens * a.packs;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kBlock; i0 < all;
       i0 += static_cast<int64_t>(gridDim.x) * kBlock) {
    // the workgroup's first token and pack, then 32-bit steps from there
    const int64_t t0 = all >> 32 == 0 ? static_cast<uint32_t>(i0) / a.packs : i0 / a.packs;
    const uint32_t k = static_cast<uint32_t>(i0 - t0 * a.packs) + threadIdx.x;
    const uint32_t step = row_step(a, k), c = (k - step * a.packs) * V;
    const int64_t t = t0 + step;
    const int n = static_cast<int>(a.cols - c);
    if (t >= a.tokens) continue;
    const int64_t r = row_of(ld_id<WIDE>(a.ids, t), a.first_row, a.rows);
    const int64_t p = POS ? row_of(ld_id<WIDE>(a.pos_ids, t), 0, a.pos_rows) : -1;
    Held<V, TDT> f{}, g{};
    if (r >= 0) f = ld_held<V, TDT, WHOLE>(a.table + r * a.cols * kSize<TDT>, c, a.cols);
    if (p >= 0) g = ld_held<V, TDT, WHOLE>(a.pos_table + p * a.cols * kSize<TDT>, c, a.cols);
    settle_held<V, TDT, WHOLE>(f, c, a.cols);
    if constexpr (POS) settle_held<V, TDT, WHOLE>(g, c, a.cols);
    float y[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      y[i] = r >= 0 ? held(f, i) * a.scale : 0.0f;  // +0, whatever the scale
      if constexpr (POS) y[i] = y[i] + (p >= 0 ? held(g, i) : -0.0f);  // -0 adds nothing
    }
    st_some<DT, WHOLE>(reinterpret_cast<char*>(a.y.at + t * a.y.pitch) + c * kSize<DT>, n, narrow<DT>(y));
  }
}

// ---- the tokens in the order of their rows ------------------------------------

struct SortArgs {
  const void* ids;
  TokenRow* list;     // the outcome
  TokenRow* other;    // before or after a pass
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

// Zeros by workgroup i of n, clear_groups(bytes, WG): 16 bytes per lane, which ends.
// 1.05 GB 154 us, 6.8 TB/s; 177 to 185 with workgroups that stay (4 or 8 stores
// of a lane at a time, 16 or 32 waves per CU), 179 with four stores per lane that
// ends, 158 with non-temporal stores; 77 MB 11.1 to 14.4 us in the same order.
template <int WG>
__device__ __forceinline__ void clear_part(char* at, int64_t bytes, int64_t i, int64_t n) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(at), hi = lo + bytes;
  for (uintptr_t to = (lo & ~uintptr_t{15}) + 16 * (i * WG + threadIdx.x); to < hi; to += 16 * WG * n) {
    if (to >= lo && to + 16 <= hi) {
      *reinterpret_cast<u32x4a16*>(to) = u32x4a16{0, 0, 0, 0};
    } else {  // the ends
      for (int k = 0; k < 16; k += 2)
        if (to + k >= lo && to + k < hi) *reinterpret_cast<uint16_t*>(to + k) = 0;
    }
  }
}
// As many as the bytes need; fewer where a launch cannot count them.
int64_t clear_groups(int64_t bytes, int lanes) {
  const int64_t groups = (bytes + 15 + 16 * lanes - 1) / (16 * lanes);
  const int64_t most = kMaxGroups / (lanes / kBlock) - 4096;
  return groups < most ? groups : most;
}

// Lanes of the wave whose digit is this lane's, of those that are live.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, bool live, int bits) {
  const uint64_t all = __ballot(live);
  uint32_t lo = static_cast<uint32_t>(all), hi = static_cast<uint32_t>(all >> 32);
  for (int b = 0; b < bits; ++b) {
    const uint32_t set = 0u - ((digit >> b) & 1u);
    const uint64_t with = __ballot(set != 0);
    lo &= ~(static_cast<uint32_t>(with) ^ set);
    hi &= ~(static_cast<uint32_t>(with >> 32) ^ set);
  }
  return lo | static_cast<uint64_t>(hi) << 32;
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

// One launch: each of kBuckets workgroups sorts the tokens whose row is its number,
// modulo kBuckets, and the other workgroups clear.  Rows need to stay together, not
// to be in order, so the list is bucket after bucket, each in the order of row /
// kBuckets.  Every sorting workgroup goes through all tokens twice: first to count
// those of the buckets before its own, then to take its own.  Up to kFew of these
// it sorts by comparing each with all; more in radix passes, in which each
// wave has a run of them and a count per digit, and sums over digits and waves turn
// the counts into the places of each wave's tokens.
constexpr int kBuckets = 64;
// Tokens that are sorted by comparison at most: a bucket of 620 of them (8192 in all)
// takes 5 us longer so than in passes, one of 310 (4096 in all) no longer.
constexpr int kFew = 512;
// Where all workgroups go through all tokens, their time grows with these: 2048, 4096,
// 8192 and 16384 tokens 6, 8.5, 11.5 and 19 us; 131072 97, where the passes below
// take 25.  All of the gradient with this sort and with the passes, us: 2048 x 64,
// added to 50257 rows, 15.5 / 23.6, 8192 20.7 / 28.8, 12288 26.3 / 32.3, 16384 29.2 /
// 29.4, 16384 x 768 35.5 / 31.4.
constexpr int kIdSteps = 8;  // steps of 64 tokens whose ids a wave loads together

// A wave's run of the tokens; the rows of its first kIdSteps steps stay in registers.
struct IdRun {
  int t0, t1;
  uint32_t row[kIdSteps];
};
template <bool WIDE>
__device__ __forceinline__ void ld_ids(const SortArgs& a, int t, int t1, uint32_t (&row)[kIdSteps]) {
#pragma unroll
  for (int k = 0; k < kIdSteps; ++k) {
    const int x = t + k * kWave + static_cast<int>(threadIdx.x % kWave);
    row[k] = x < t1 ? ld_row_of<WIDE>(a, x) : static_cast<uint32_t>(a.rows);
  }
}
// Calls f(row, token) for the steps of the run, and for what the last has beyond the
// run, as tokens without a row.
template <bool WIDE, class F>
__device__ __forceinline__ void for_ids(const SortArgs& a, const IdRun& ids, F&& f) {
  const int lane = threadIdx.x % kWave;
  if (ids.t0 >= ids.t1) return;
#pragma unroll
  for (int k = 0; k < kIdSteps; ++k) f(ids.row[k], ids.t0 + k * kWave + lane);
  for (int t = ids.t0 + kIdSteps * kWave; t < ids.t1; t += kIdSteps * kWave) {
    uint32_t row[kIdSteps];
    ld_ids<WIDE>(a, t, ids.t1, row);
#pragma unroll
    for (int k = 0; k < kIdSteps; ++k) f(row[k], t + k * kWave + lane);
  }
}

template <bool WIDE, int LANES>
__global__ __launch_bounds__(LANES) void sort_buckets_kernel(SortArgs a) {
  constexpr int kWaves = LANES / kWave;
  __shared__ uint32_t counts[kWaves << kBucketBits];
  __shared__ uint32_t work[kWaves];
  __shared__ uint32_t found[3][kWaves];
  __shared__ TokenRow few[kFew];
  __shared__ u32x4a16 keys[kFew / 4];
  if (blockIdx.x >= kBuckets) {
    clear_part<LANES>(a.clear, a.clear_bytes, static_cast<int64_t>(blockIdx.x) - kBuckets,
                      gridDim.x - kBuckets);
    return;
  }
  const uint32_t bucket = blockIdx.x, none = static_cast<uint32_t>(a.rows);
  if (bucket == 0 && threadIdx.x == 0) *a.long_rows = 0;
  const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint64_t below = (uint64_t{1} << lane) - 1;
  const int each = (a.tokens + LANES - 1) / LANES * kWave;
  IdRun ids;
  ids.t0 = wave * each;
  ids.t1 = ids.t0 + each < a.tokens ? ids.t0 + each : a.tokens;
  ld_ids<WIDE>(a, ids.t0, ids.t1, ids.row);
  uint32_t own = 0, less = 0, some = 0;
  for_ids<WIDE>(a, ids, [&](uint32_t row, int) {
    own += __popcll(__ballot(row != none && row % kBuckets == bucket));
    less += __popcll(__ballot(row != none && row % kBuckets < bucket));
    some += __popcll(__ballot(row != none));
  });
  if (lane == 0) {
    found[0][wave] = own;
    found[1][wave] = less;
    found[2][wave] = some;
  }
  if (threadIdx.x < kFew) keys[threadIdx.x / 4][threadIdx.x % 4] = ~0u;
  __syncthreads();
  uint32_t first = 0, before = 0, count = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += found[0][w];
    count += found[0][w];
    first += found[1][w];
    all += found[2][w];
  }
  // behind the last token that has a row
  for (uint32_t p = all + bucket * LANES + threadIdx.x; p < static_cast<uint32_t>(a.tokens);
       p += kBuckets * LANES)
    a.list[p] = TokenRow{none, 0};
  if (count <= kFew) {
    uint32_t place = before;
    for_ids<WIDE>(a, ids, [&](uint32_t row, int t) {
      const bool mine = row != none && row % kBuckets == bucket;
      const uint64_t m = __ballot(mine);
      if (mine) {
        const uint32_t p = place + __popcll(m & below);
        few[p] = TokenRow{row, static_cast<uint32_t>(t)};
        keys[p / 4][p % 4] = row;
      }
      place += __popcll(m);
    });
    __syncthreads();
    if (threadIdx.x >= count) return;
    // before it: smaller rows, and the same row's earlier tokens
    const TokenRow q = few[threadIdx.x];
    uint32_t p = 0;
    for (uint32_t i = 0; i < (count + 3) / 4; ++i) {
      const u32x4a16 k = keys[i];
      const uint32_t bound = q.row + (i < threadIdx.x / 4);
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) p += k[j] < bound;
    }
    const u32x4a16 k = keys[threadIdx.x / 4];
#pragma unroll
    for (uint32_t j = 0; j < 3; ++j) p += k[j] == q.row && j < threadIdx.x % 4;
    a.list[first + p] = q;
    return;
  }
  TokenRow* from = (a.passes % 2 ? a.other : a.list) + first;
  TokenRow* to = (a.passes % 2 ? a.list : a.other) + first;
  uint32_t place = before;
  for_ids<WIDE>(a, ids, [&](uint32_t row, int t) {
    const bool mine = row != none && row % kBuckets == bucket;
    const uint64_t m = __ballot(mine);
    if (mine) from[place + __popcll(m & below)] = TokenRow{row, static_cast<uint32_t>(t)};
    place += __popcll(m);
  });
  __syncthreads();
  const int digits = 1 << a.bits;
  uint32_t* mine = counts + wave * digits;
  const uint32_t run = (count + LANES - 1) / LANES * kWave;
  const uint32_t t0 = wave * run, t1 = t0 + run < count ? t0 + run : count;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
    for (int i = threadIdx.x; i < kWaves * digits; i += LANES) counts[i] = 0;
    __syncthreads();
    for (uint32_t t = t0 + lane; t < t1; t += kWave)
      atomicAdd(mine + ((from[t].row / kBuckets >> shift) & (digits - 1)), 1u);
    __syncthreads();
    const int d = threadIdx.x;
    uint32_t n[kWaves], sum = 0, total;
    if (d < digits) {
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        n[w] = counts[w * digits + d];
        sum += n[w];
      }
    }
    uint32_t at = scan_lanes<LANES>(sum, work, &total);
    if (d < digits) {
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        counts[w * digits + d] = at;
        at += n[w];
      }
    }
    __syncthreads();
    for (uint32_t t = t0; t < t1; t += kWave) {
      const bool live = t + lane < t1;
      TokenRow q{0, 0};
      if (live) q = from[t + lane];
      const uint32_t p = take_place(mine, (q.row / kBuckets >> shift) & (digits - 1), live, a.bits, lane);
      if (live) to[p] = q;
    }
    __syncthreads();
    TokenRow* x = from;
    from = to;
    to = x;
  }
}
static_assert(1 << kBucketBits <= 512 && kFew <= 512, "a digit or a token per lane");

// More tokens, several launches: each workgroup has a tile of the tokens, and each of
// its waves a run of the tile.  Two kernels per pass: one counts the tiles' digits,
// the other adds up the counts before its tile and digit and puts the tokens in
// their places.  Short tiles, so that many waves wait at once: all of the gradient
// of 131072 tokens 107 us with tiles of 1024, 108 with 2048, 117 with 4096; of
// 32768 49, 53 and 65.
constexpr int kTileLanes = 512, kTileWaves = kTileLanes / kWave;
constexpr int kTileSteps = 2;  // of 64 tokens, that a wave loads together

// Calls f(row and token, whether they are there) for the steps of a wave's run of the
// tile.
template <bool WIDE, bool FIRST, class F>
__device__ __forceinline__ void for_run(const SortArgs& a, const TokenRow* from, F&& f) {
  constexpr int K = kTileSteps;
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
__global__ __launch_bounds__(kTileLanes) void sort_count_kernel(SortArgs a, const TokenRow* from,
                                                               int shift, int tiles) {
  if (static_cast<int>(blockIdx.x) >= tiles) {
    clear_part<kTileLanes>(a.clear, a.clear_bytes, static_cast<int64_t>(blockIdx.x) - tiles,
                           gridDim.x - tiles);
    return;
  }
  __shared__ uint32_t counts[1 << kSortBits];
  if (FIRST && blockIdx.x == 0 && threadIdx.x == 0) *a.long_rows = 0;
  const int digits = 1 << a.bits;
  for (int i = threadIdx.x; i < digits; i += kTileLanes) counts[i] = 0;
  __syncthreads();
  for_run<WIDE, FIRST>(a, from, [&](TokenRow q, bool live) {
    if (live) atomicAdd(counts + ((q.row >> shift) & (digits - 1)), 1u);
  });
  __syncthreads();
  for (int i = threadIdx.x; i < digits; i += kTileLanes) a.counts[(blockIdx.x << a.bits) + i] = counts[i];
}

template <bool WIDE, bool FIRST>
__global__ __launch_bounds__(kTileLanes) void sort_place_kernel(SortArgs a, const TokenRow* from,
                                                               TokenRow* to, int shift) {
  __shared__ uint32_t counts[kTileWaves << kSortBits];
  __shared__ uint32_t work[kTileWaves];
  const int digits = 1 << a.bits;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  uint32_t* mine = counts + wave * digits;
  for (int i = threadIdx.x; i < kTileWaves * digits; i += kTileLanes) counts[i] = 0;
  __syncthreads();
  for_run<WIDE, FIRST>(a, from, [&](TokenRow q, bool live) {
    if (live) atomicAdd(mine + ((q.row >> shift) & (digits - 1)), 1u);
  });
  __syncthreads();
  uint32_t carry = 0;
  for (int d0 = 0; d0 < digits; d0 += kTileLanes) {
    const int d = d0 + threadIdx.x;
    uint32_t sum = 0, before = 0, all;
    if (d < digits) {
      const uint32_t* at = a.counts + d;
      const int tiles = gridDim.x, own = blockIdx.x;
#pragma unroll 16
      for (int t = 0; t < tiles; ++t) {
        const uint32_t n = at[t << a.bits];
        sum += n;
        if (t < own) before += n;
      }
    }
    uint32_t place = carry + scan_lanes<kTileLanes>(sum, work, &all) + before;
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

// V columns of a row of the gradient, n of them there; old: what it holds.
template <int V, int GDT, bool ADD, bool WHOLE>
__device__ __forceinline__ void st_grad(const SumArgs& a, int64_t row, int c, int n, const Vals<V>& sum,
                                        Held<V, GDT> old) {
  Vals<V> f;
  if constexpr (ADD) settle_held<V, GDT, WHOLE>(old, c, a.cols);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    f.v[i] = sum.v[i] * a.scale;
    if constexpr (ADD) f.v[i] = held(old, i) + f.v[i];
  }
  st_vals<V, GDT, WHOLE>(static_cast<char*>(a.grad) + (row * a.cols + c) * kSize<GDT>, n, f);
}
template <int V, int GDT, bool ADD, bool WHOLE>
__device__ __forceinline__ Held<V, GDT> ld_grad(const SumArgs& a, int64_t row, int c) {
  if constexpr (ADD)
    return ld_held<V, GDT, WHOLE>(static_cast<const char*>(a.grad) + row * a.cols * kSize<GDT>, c, a.cols);
  return Held<V, GDT>{};
}

// V sums, n of them there, through the cache: the next kernel reads them.
template <int V, bool WHOLE>
__device__ __forceinline__ void st_sums(float* to, int n, const Vals<V>& x) {
#pragma unroll
  for (int k = 0; k < V / 4; ++k) {
    if (n >= 4 * k + 4) {
      *reinterpret_cast<f32x4*>(to + 4 * k) =
          f32x4{x.v[4 * k], x.v[4 * k + 1], x.v[4 * k + 2], x.v[4 * k + 3]};
    } else if (!WHOLE) {
#pragma unroll
      for (int i = 4 * k; i < 4 * k + 4; ++i)
        if (i < n) to[i] = x.v[i];
    }
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

// A window is W places of the sorted list.  The wave of a window and slab of
// columns (1 KiB of dy's; of narrower rows some lanes have none) sums every table row
// whose tokens begin in the window, as far as they go, if they are at most W.  The
// tokens of a row that has more (a long row) are summed by each window that they
// meet: where they begin, to the window's second row of sums, elsewhere to its first;
// sum_join_kernel adds these.
//
// What is where shows in masks of the 3 * W places from W before the
// window's first: bit l of `on` says that place l holds the row of place l - 1.
//
// Short windows where the tokens are few, so that there are more waves with less to
// do one after the other (us with 8 and 16: 500 x 768, added to, 15.2 / 18.4; 2048 x
// 768 21.1 / 25.1; 8192 x 768 48.1 / 50.3), long ones elsewhere, which leave half
// the parts of sums (32768 x 768 66.2 / 59.0; 131072 x 1024 147 / 120).
constexpr int kWindowFew = 8, kWindowMany = 16;
constexpr int64_t kWindowElems = int64_t{1} << 23;

struct Window {
  uint32_t row, token;  // of place `lane`
  uint64_t on, live;
};
template <int W>
__device__ __forceinline__ Window ld_window(const SumArgs& a, int64_t w, int lane) {
  const int64_t p = (w - 1) * W + lane;
  const uint32_t none = static_cast<uint32_t>(a.rows);
  TokenRow q{none, 0};
  if (lane < 3 * W && p >= 0 && p < a.tokens) q = a.list[p];
  const uint32_t before = __shfl_up(q.row, 1, kWave);
  Window x;
  x.row = q.row;
  x.token = q.token;
  x.live = __ballot(q.row != none);
  x.on = __ballot(lane > 0 && q.row == before) & x.live;
  return x;
}
// Whether the row that begins at place s has more than W tokens.
template <int W>
__device__ __forceinline__ bool is_long(uint64_t on, int s) {
  constexpr uint64_t all = (uint64_t{1} << W) - 1;
  return ((on >> (s + 1)) & all) == all;
}
// The last place up to l at which a row begins; 0: at none from 1 on.
__device__ __forceinline__ int begin_of(uint64_t on, int l) {
  const uint64_t begins = ~on & ((uint64_t{2} << l) - 2);
  return begins ? 63 - __builtin_clzll(begins) : 0;
}

template <int W, int DT, int GDT, bool ADD, bool STREAM, bool WHOLE>
__device__ __forceinline__ void sum_unit(const SumArgs& a, int64_t unit) {
  constexpr int V = kPack<DT>;
  const int lane = threadIdx.x % kWave;
  const int64_t w = unit / a.slabs;
  const int slab = static_cast<int>(unit - w * a.slabs);
  const int c = (slab * kWave + lane) * V, n = a.cols - c;
  const Window x = ld_window<W>(a, w, lane);
  const uint64_t stop = ~x.on;
  int l = W;
  bool head = false;  // a long row that began before the window
  if (x.on >> l & 1) {
    const int s = begin_of(x.on, l);
    head = s == 0 || is_long<W>(x.on, s);
    if (!head) l += __builtin_ctzll(stop >> l);  // its own window's
  }
  int end = 2 * W;
  bool tail = false;
  if (x.on >> end & 1) {
    const int s = begin_of(x.on, end);
    if (s >= W) {  // or it is the head, which meets all of the window
      tail = is_long<W>(x.on, s);
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
  // rows of dy in flight per wave, and of the gradient that are added to
  constexpr int kLoads = 8;
  for (; l < end; l += kLoads) {
    Pack<DT> p[kLoads];
    Held<V, GDT> old[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      if (l + u >= end) break;
      const uint32_t t = __builtin_amdgcn_readlane(x.token, l + u);
      p[u] = ld_some<DT, WHOLE, STREAM>(reinterpret_cast<const char*>(a.dy.at + t * a.dy.pitch), c,
                                        a.cols);
      if (ADD && !(x.on >> (l + u + 1) & 1))
        old[u] = ld_grad<V, GDT, ADD, WHOLE>(a, __builtin_amdgcn_readlane(x.row, l + u), c);
    }
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      if (l + u >= end) break;
      float f[V];
      settle<DT, WHOLE>(p[u], c, a.cols);
      widen<DT>(p[u], f);
#pragma unroll
      for (int i = 0; i < V; ++i) sum.v[i] = sum.v[i] + f[i];
      const bool last = l + u + 1 == end;
      if (!last && (x.on >> (l + u + 1) & 1)) continue;
      const bool part = head || (last && tail);
      if (part) {
        float* to = a.partial + (2 * w + (head ? 0 : 1)) * a.cols + c;
        st_sums<V, WHOLE>(to, n, sum);
      } else {
        st_grad<V, GDT, ADD, WHOLE>(a, __builtin_amdgcn_readlane(x.row, l + u), c, n, sum, old[u]);
      }
      head = false;
#pragma unroll
      for (int i = 0; i < V; ++i) sum.v[i] = 0.0f;
    }
  }
}

template <int W, int DT, int GDT, bool ADD, bool STREAM, bool WHOLE>
__global__ __launch_bounds__(kBlock) void sum_kernel(SumArgs a) {
  for_units(static_cast<int64_t>(a.windows) * a.slabs,
            [&](int64_t unit) { sum_unit<W, DT, GDT, ADD, STREAM, WHOLE>(a, unit); });
}

// A long row's sum: a workgroup per row and 256 columns, whose waves take equal
// shares of its windows' sums.  131072 tokens of 1024 columns, 6e2 long rows, the
// longest of 490 windows: 17 us, of which 37 MB of sums are a third; the rest is a
// chain of five dependent loads per row.  Four waves 22 us, sixteen 26; a wave to a
// row of at most 16 windows, and a workgroup to others, 16 here and 8 for 5 with
// 8192 tokens.
constexpr int kJoinV = 4, kJoinSlab = kWave * kJoinV, kJoinLoads = 8, kJoinWaves = 8;

template <int W, int GDT, bool ADD, bool WHOLE>
__global__ __launch_bounds__(kJoinWaves * kWave) void sum_join_kernel(SumArgs a) {
  __shared__ Vals<kJoinV> sums[kJoinWaves][kWave];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t units = static_cast<int64_t>(a.long_rows[0]) * a.slabs;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int64_t k = unit / a.slabs, w = a.long_rows[1 + k];
    const int c = (static_cast<int>(unit - k * a.slabs) * kWave + lane) * kJoinV, n = a.cols - c;
    const uint32_t row = a.list[(w + 1) * W].row;
    Held<kJoinV, GDT> old{};
    if (wave == 0) old = ld_grad<kJoinV, GDT, ADD, WHOLE>(a, row, c);
    int64_t more = 1;  // windows after w that it meets
    // of the next 64, or of each 64th, those up to the first that it does not meet
    const auto meets = [&](int64_t step) -> int64_t {
      const int64_t x = (w + 1 + more + step * lane) * W;
      const uint64_t stops = ~__ballot(x < a.tokens && a.list[x < a.tokens ? x : 0].row == row);
      return stops ? __builtin_ctzll(stops) : kWave;
    };
    while (true) {
      const int64_t near = meets(1);
      more += near;
      if (near < kWave) break;
      const int64_t far = meets(kWave);
      if (far > 0) more += (far - 1) * kWave + 1;
    }
    // rows of sums 2 w + 1, 2 (w + 1), 2 (w + 2) ...
    const int64_t each = (more + kJoinWaves) / kJoinWaves;
    const int64_t i1 = (wave + 1) * each < more + 1 ? (wave + 1) * each : more + 1;
    Vals<kJoinV> sum;
#pragma unroll
    for (int i = 0; i < kJoinV; ++i) sum.v[i] = 0.0f;
    for (int64_t i = wave * each; i < i1; i += kJoinLoads) {
      Held<kJoinV, kF32> f[kJoinLoads];
#pragma unroll
      for (int u = 0; u < kJoinLoads; ++u) {
        const int64_t at = i + u == 0 ? 2 * w + 1 : 2 * (w + i + u);
        f[u] = Held<kJoinV, kF32>{};
        if (i + u < i1)
          f[u] = ld_held<kJoinV, kF32, WHOLE>(reinterpret_cast<const char*>(a.partial + at * a.cols), c,
                                              a.cols);
      }
#pragma unroll
      for (int u = 0; u < kJoinLoads; ++u) {
        settle_held<kJoinV, kF32, WHOLE>(f[u], c, a.cols);
#pragma unroll
        for (int q = 0; q < kJoinV; ++q) sum.v[q] = sum.v[q] + held(f[u], q);
      }
    }
    sums[wave][lane] = sum;
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int i = 1; i < kJoinWaves; ++i)
#pragma unroll
        for (int q = 0; q < kJoinV; ++q) sum.v[q] = sum.v[q] + sums[i][lane].v[q];
      st_grad<kJoinV, GDT, ADD, WHOLE>(a, row, c, n, sum, old);
    }
    __syncthreads();
  }
}

int bits_of(uint64_t x) { return x == 0 ? 0 : 64 - __builtin_clzll(x); }

size_t up256(size_t x) { return (x + 255u) & ~static_cast<size_t>(255u); }

// Tokens per tile: no more tiles than kTilesMost, so that each may add up the
// counts of all.
constexpr int kTilesMost = 256, kTileStep = kTileLanes * kTileSteps;
int64_t tile_of(int64_t tokens) {
  const int64_t steps = (tokens + kTileStep - 1) / kTileStep;
  return (steps + kTilesMost - 1) / kTilesMost * kTileStep;
}

int window_of(int64_t tokens, int64_t cols) {
  return tokens * cols <= kWindowElems ? kWindowFew : kWindowMany;
}

}  // namespace

EmbedLayout embed_layout(int64_t tokens, int64_t cols) {
  EmbedLayout l;
  const size_t list = up256(sizeof(TokenRow) * static_cast<size_t>(tokens));
  const size_t windows = static_cast<size_t>((tokens - 1) / window_of(tokens, cols) + 1);
  const size_t tiles =
      tokens <= kSortAlone ? 0 : static_cast<size_t>((tokens - 1) / tile_of(tokens) + 1);
  l.list = 0;
  l.other = list;
  l.counts = l.other + list;
  l.long_rows = l.counts + (sizeof(uint32_t) << kSortBits) * tiles;
  l.partial = l.long_rows + up256(sizeof(uint32_t) * (windows + 1));
  l.total = l.partial + up256(sizeof(float) * 2 * windows * static_cast<size_t>(cols));
  return l;
}

// The layout grows with the tokens, but for steps down where windows get longer (few
// tokens are the most before) and where tiles do (every multiple of kTiles tokens is).
size_t embed_workspace(int64_t tokens, int64_t cols) {
  constexpr int64_t kTiles = int64_t{kTilesMost} * kTileStep;
  const int64_t few = kWindowElems / cols < tokens ? kWindowElems / cols : tokens;
  size_t most = 0;
  for (const int64_t t : {tokens, tokens / kTiles * kTiles, few, few / kTiles * kTiles}) {
    const size_t bytes = t > 0 ? embed_layout(t, cols).total : 0;
    if (bytes > most) most = bytes;
  }
  return most;
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
    a.inverse = static_cast<uint32_t>(((uint64_t{1} << 32) + a.packs - 1) / a.packs);
    const int64_t groups = (L.tokens * a.packs + kBlock - 1) / kBlock;
    const dim3 grid(static_cast<unsigned>(groups < kMaxGroups ? groups : kMaxGroups));
    with_gdt(L.tdt, [&](auto t) {
      constexpr int TDT = decltype(t)::value;
      const auto go = [&](auto wide, auto pos) {
        constexpr bool WIDE = decltype(wide)::value != 0, POS = decltype(pos)::value != 0;
        if (a.cols % kPack<DT> == 0) embed_kernel<DT, TDT, WIDE, POS, true><<<grid, kBlock, 0, L.stream>>>(a);
        else embed_kernel<DT, TDT, WIDE, POS, false><<<grid, kBlock, 0, L.stream>>>(a);
      };
      const auto pick = [&](auto wide) { L.pos_table ? go(wide, IC<1>{}) : go(wide, IC<0>{}); };
      L.wide_ids ? pick(IC<1>{}) : pick(IC<0>{});
    });
  });
  return hipGetLastError();
}

namespace {

// Where clearing takes longer than sorting, its workgroups are small (128256 x 4096
// bf16 212 us in all, with 1024 lanes 222); else the sort's are large (50257 x 768
// 27 us, with 512 lanes 33).
constexpr int64_t kClearLong = int64_t{256} << 20;

// Up to so many bytes, dy may still be in the 256 MB cache where its rows are added to
// a gradient, and is read through it (us through it and past it: 16384 x 1024 37.3 /
// 39.9, 4096 x 4096 28.1 / 31.0, 32768 x 768 42.3 / 43.8, 131072 x 1024 122 / 106).
// Into a gradient that was cleared before it is read past it: a large one has filled
// the cache (16384 x 1024 52.0 / 43.3, 32768 x 768 53.2 / 49.1), and small ones gain
// more by it than they lose (a position table's: 8192 x 768 into 1024 rows 15.2 / 13.4,
// 32768 x 768 into 1024 rows 43.9 / 45.7, 16384 x 4096 into 8192 rows 66.9 / 58.3;
// 8192 x 768 into 2000 rows 24.6 / 24.4).
constexpr int64_t kSumCached = int64_t{64} << 20;
static_assert(kWindowElems * 4 <= kSumCached, "few tokens' rows are read through it");

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
  a.clear = static_cast<char*>(L.grad);
  a.clear_bytes = L.rows * L.cols * (L.gdt == kF32 ? 4 : 2);
  const auto digits = [&](int key_bits, int most) {
    a.passes = (key_bits + most - 1) / most;
    a.bits = a.passes ? (key_bits + a.passes - 1) / a.passes : 0;
  };
  if (L.tokens <= kSortAlone) {
    digits(bits_of(static_cast<uint64_t>(L.rows - 1) / kBuckets), kBucketBits);
    const auto go = [&](auto lanes) {
      constexpr int LANES = decltype(lanes)::value;
      const int64_t clearers = L.accumulate ? 0 : clear_groups(a.clear_bytes, LANES);
      const dim3 grid(static_cast<unsigned>(kBuckets + clearers));
      if (L.wide_ids) sort_buckets_kernel<true, LANES><<<grid, LANES, 0, L.stream>>>(a);
      else sort_buckets_kernel<false, LANES><<<grid, LANES, 0, L.stream>>>(a);
    };
    if (!L.accumulate && a.clear_bytes > kClearLong) go(IC<512>{});
    else go(IC<1024>{});
    return hipGetLastError();
  }
  const int64_t clearers = L.accumulate ? 0 : clear_groups(a.clear_bytes, kTileLanes);
  digits(bits_of(static_cast<uint64_t>(L.rows)), kSortBits);  // a row, or rows itself
  a.tile = static_cast<int32_t>(tile_of(L.tokens));
  const int tiles = static_cast<int>((L.tokens + a.tile - 1) / a.tile);
  const TokenRow* from = nullptr;
  TokenRow* to = a.passes % 2 ? a.list : a.other;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
    const dim3 grid(static_cast<unsigned>(tiles)), first(static_cast<unsigned>(tiles + clearers));
    if (pass > 0) {
      sort_count_kernel<false, false><<<grid, kTileLanes, 0, L.stream>>>(a, from, shift, tiles);
      sort_place_kernel<false, false><<<grid, kTileLanes, 0, L.stream>>>(a, from, to, shift);
    } else if (L.wide_ids) {
      sort_count_kernel<true, true><<<first, kTileLanes, 0, L.stream>>>(a, from, shift, tiles);
      sort_place_kernel<true, true><<<grid, kTileLanes, 0, L.stream>>>(a, from, to, shift);
    } else {
      sort_count_kernel<false, true><<<first, kTileLanes, 0, L.stream>>>(a, from, shift, tiles);
      sort_place_kernel<false, true><<<grid, kTileLanes, 0, L.stream>>>(a, from, to, shift);
    }
    from = to;
    to = to == a.list ? a.other : a.list;
  }
  return hipGetLastError();
}

__global__ __launch_bounds__(kBlock) void clear_kernel(char* at, int64_t bytes) {
  clear_part<kBlock>(at, bytes, blockIdx.x, gridDim.x);
}

}  // namespace

hipError_t launch_embed_grad(const EmbedGradLaunch& L) {
  if (L.tokens == 0) {
    const int64_t bytes = L.rows * L.cols * (L.gdt == kF32 ? 4 : 2);
    clear_kernel<<<dim3(static_cast<unsigned>(clear_groups(bytes, kBlock))), kBlock, 0, L.stream>>>(
        static_cast<char*>(L.grad), bytes);
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
  const int window = window_of(L.tokens, L.cols);
  a.windows = static_cast<int32_t>((L.tokens - 1) / window + 1);
  a.cols = L.cols;
  a.scale = L.scale;
  with_gdt(L.gdt, [&](auto g) {
    constexpr int GDT = decltype(g)::value;
    const auto go = [&](auto add, auto window) {
      constexpr int W = decltype(window)::value;
      constexpr bool ADD = decltype(add)::value != 0;
      with_gdt(L.dt, [&](auto d) {
        constexpr int DT = decltype(d)::value, kSlab = kWave * kPack<DT>;
        a.slabs = (L.cols + kSlab - 1) / kSlab;
        const int64_t groups = (static_cast<int64_t>(a.windows) * a.slabs + kWaves - 1) / kWaves;
        const dim3 grid(static_cast<unsigned>(groups < kMaxGroups ? groups : kMaxGroups));
        const auto sum = [&](auto whole) {
          constexpr bool WHOLE = decltype(whole)::value != 0;
          if constexpr (ADD) {
            if (W == kWindowFew || L.tokens * L.cols * kSize<DT> <= kSumCached) {
              sum_kernel<W, DT, GDT, ADD, false, WHOLE><<<grid, kBlock, 0, L.stream>>>(a);
              return;
            }
          }
          if constexpr (!ADD || W == kWindowMany)
            sum_kernel<W, DT, GDT, ADD, true, WHOLE><<<grid, kBlock, 0, L.stream>>>(a);
        };
        L.cols % kPack<DT> == 0 ? sum(IC<1>{}) : sum(IC<0>{});
      });
      if (L.tokens <= W) return;  // no long row
      a.slabs = (L.cols + kJoinSlab - 1) / kJoinSlab;
      const int64_t most = int64_t{cu_count()} * (32 / kJoinWaves);
      const int64_t units = L.tokens / (W + 1) * a.slabs;
      const dim3 grid(static_cast<unsigned>(units < most ? units : most));
      if (L.cols % kJoinV == 0)
        sum_join_kernel<W, GDT, ADD, true><<<grid, kJoinWaves * kWave, 0, L.stream>>>(a);
      else
        sum_join_kernel<W, GDT, ADD, false><<<grid, kJoinWaves * kWave, 0, L.stream>>>(a);
    };
    const auto pick = [&](auto w) { L.accumulate ? go(IC<1>{}, w) : go(IC<0>{}, w); };
    window == kWindowFew ? pick(IC<kWindowFew>{}) : pick(IC<kWindowMany>{});
  });
  return hipGetLastError();
}

}  // namespace zs
