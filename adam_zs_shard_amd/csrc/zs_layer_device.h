// zs_layer_device.h -- device code shared by the layer kernels: 16 bytes of a
// row at a time, and sums over a wave.
#pragma once

#include "zs_adamw_device.h"
#include "zs_layer.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

// Elements in 16 bytes of a row.
template <int DT>
constexpr int kPack = DT == kF32 ? 4 : 8;

template <int DT>
struct Pack {
  std::conditional_t<DT == kF32, f32x4, u32x4> x;
};

typedef uint32_t Word __attribute__((aligned(2)));

template <int V>
struct Vals {
  float v[V];
};

// Elements c .. c + V - 1 of a row of cols, as they are held; beyond the row zeros.
// A row's last elements, if they are fewer than V, come with a load of the row's last
// V, and settle_held() puts them first and zeros behind them, after all loads of a
// lane are on their way.  Element by element they were up to V - 1 loads that waited
// for one another: norms' backward pass, 742 x 1043 fp16 16.3 us, now 9.5, 20,000 x
// 1001 bf16 46.6 / 35.8; the table's gradient, 43,231 x 1017 bf16 65.6 / 55.5.
// STREAM: non-temporal.  WHOLE: cols is a multiple of V, and there is nothing to settle.
template <int V, int DT>
struct Held {
  uint32_t x[V * kSize<DT> / 4];
};
template <int V, int DT, bool WHOLE = false, bool STREAM = false>
__device__ __forceinline__ Held<V, DT> ld_held(const char* row, int c, int cols) {
  constexpr int N = V * kSize<DT> / 4;
  Held<V, DT> h{};
  if (c >= cols) return h;
  if (!WHOLE && cols < V) {  // c is 0
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < cols) {
        if constexpr (DT == kF32)
          h.x[i] = reinterpret_cast<const uint32_t*>(row)[i];
        else
          h.x[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(row)[i]) << (16 * (i % 2));
      }
    return h;
  }
  const char* at = row + static_cast<int64_t>(WHOLE || c + V <= cols ? c : cols - V) * kSize<DT>;
  if constexpr (N == 2) {
    const u32x2 q = *reinterpret_cast<const u32x2*>(at);
    h.x[0] = q[0];
    h.x[1] = q[1];
  } else {
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
      const auto* p = reinterpret_cast<const u32x4*>(at) + k;
      const u32x4 q = STREAM ? __builtin_nontemporal_load(p) : *p;
#pragma unroll
      for (int i = 0; i < 4; ++i) h.x[4 * k + i] = q[i];
    }
  }
  return h;
}
template <int V, int DT, bool WHOLE = false>
__device__ __forceinline__ void settle_held(Held<V, DT>& h, int c, int cols) {
  if constexpr (WHOLE) return;
  constexpr int N = V * kSize<DT> / 4;
  const int back = c + V - cols;
  if (back <= 0 || back >= V || cols < V) return;
  const int halves = back * kSize<DT> / 2;  // of a word, to move down
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t up = i + 1 < N ? h.x[i + 1] : 0u;
    h.x[i] = halves & 1 ? h.x[i] >> 16 | up << 16 : h.x[i];
  }
#pragma unroll
  for (int b = 1; b < N; b *= 2)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t up = i + b < N ? h.x[i + b] : 0u;
      h.x[i] = halves & (2 * b) ? up : h.x[i];
    }
}
template <int V, int DT>
__device__ __forceinline__ float held(const Held<V, DT>& h, int i) {
  if constexpr (DT == kF32) return __builtin_bit_cast(float, h.x[i]);
  else return i % 2 == 0 ? widen_lo<DT>(h.x[i / 2]) : widen_hi<DT>(h.x[i / 2]);
}

// The same of a pack.
template <int DT, bool WHOLE = false, bool STREAM = true>
__device__ __forceinline__ Pack<DT> ld_some(const char* row, int c, int cols) {
  return __builtin_bit_cast(Pack<DT>, ld_held<kPack<DT>, DT, WHOLE, STREAM>(row, c, cols));
}
template <int DT, bool WHOLE = false>
__device__ __forceinline__ void settle(Pack<DT>& q, int c, int cols) {
  if constexpr (!WHOLE) {
    auto h = __builtin_bit_cast(Held<kPack<DT>, DT>, q);
    settle_held(h, c, cols);
    q = __builtin_bit_cast(Pack<DT>, h);
  }
}

template <int DT>
__device__ __forceinline__ void widen(const Pack<DT>& q, float (&f)[kPack<DT>]) {
  if constexpr (DT == kF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = q.x[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = widen_lo<DT>(q.x[i]);
      f[2 * i + 1] = widen_hi<DT>(q.x[i]);
    }
  }
}
// Two values to 16 bits, each as it stands in fp32: a product that only its
// conversion to f16 uses is otherwise folded into that (v_fma_mixlo_f16), rounded
// once instead of twice and with the sign of a zero lost.
template <int DT>
__device__ __forceinline__ uint32_t narrow_pair(float lo, float hi) {
  if constexpr (DT == kF16) asm("" : "+v"(lo), "+v"(hi));
  return narrow2<DT>(lo, hi);
}
template <int DT>
__device__ __forceinline__ Pack<DT> narrow(const float (&f)[kPack<DT>]) {
  Pack<DT> q;
  if constexpr (DT == kF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) q.x[i] = f[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) q.x[i] = narrow_pair<DT>(f[2 * i], f[2 * i + 1]);
  }
  return q;
}

// The first `halves` halves of N words, fewer than all: in up to three stores.
template <int N, class T>
__device__ __forceinline__ void st_part(char* at, int halves, T x) {
  uint32_t w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = x[i];
  if constexpr (N == 4) {
    if (halves & 4) {
      __builtin_nontemporal_store(u32x2{w[0], w[1]}, reinterpret_cast<u32x2*>(at));
      w[0] = w[2];
      w[1] = w[3];
      at += 8;
    }
  }
  if (halves & 2) {
    *reinterpret_cast<Word*>(at) = w[0];
    w[0] = w[1];
    at += 4;
  }
  if (halves & 1) *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(w[0]);
}
template <int DT, bool WHOLE = false>
__device__ __forceinline__ void st_some(char* at, int n, const Pack<DT>& q) {
  if (n >= kPack<DT>) {
    __builtin_nontemporal_store(q.x, reinterpret_cast<decltype(Pack<DT>::x)*>(at));
  } else if (!WHOLE && n > 0) {
    const auto x = __builtin_bit_cast(u32x4, q.x);
    st_part<4>(at, n * (kSize<DT> / 2), x);
  }
}

// Rounds V values to `at`, n of them there.
template <int V, int DT, bool WHOLE = false>
__device__ __forceinline__ void st_vals(char* at, int n, const Vals<V>& x) {
  if constexpr (DT == kF32) {
#pragma unroll
    for (int k = 0; k < V / 4; ++k) {
      const float f[4] = {x.v[4 * k], x.v[4 * k + 1], x.v[4 * k + 2], x.v[4 * k + 3]};
      st_some<kF32, WHOLE>(at + 16 * k, n - 4 * k, narrow<kF32>(f));
    }
  } else if constexpr (V == 8) {
    st_some<DT, WHOLE>(at, n, narrow<DT>(x.v));
  } else {
    const u32x2 q{narrow_pair<DT>(x.v[0], x.v[1]), narrow_pair<DT>(x.v[2], x.v[3])};
    if (n >= 4) {
      __builtin_nontemporal_store(q, reinterpret_cast<u32x2*>(at));
    } else if (!WHOLE) {
      if (n > 0) st_part<2>(at, n, q);
    }
  }
}
// Of a vector of cols weights, from element c on; no vector: `none`.
template <int V, int WDT>
__device__ __forceinline__ Vals<V> ld_vals(const void* base, int c, int cols) {
  Held<V, WDT> h = ld_held<V, WDT>(static_cast<const char*>(base), c, cols);
  settle_held(h, c, cols);
  Vals<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.v[i] = held(h, i);
  return r;
}
template <int V>
__device__ __forceinline__ Vals<V> ld_weights(const void* base, int wdt, int c, int cols, float none) {
  Vals<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.v[i] = none;
  if (base) {
    if (wdt == kF16) r = ld_vals<V, kF16>(base, c, cols);
    else if (wdt == kBF16) r = ld_vals<V, kBF16>(base, c, cols);
    else r = ld_vals<V, kF32>(base, c, cols);
  }
  return r;
}

__device__ __forceinline__ float ld_value(const void* base, int dt, int64_t at) {
  if (dt == kF32) return static_cast<const float*>(base)[at];
  const uint16_t h = static_cast<const uint16_t*>(base)[at];
  return dt == kF16 ? widen1<kF16>(h) : widen1<kBF16>(h);
}
__device__ __forceinline__ void st_value(void* base, int dt, int64_t at, float x) {
  if (dt == kF32)
    static_cast<float*>(base)[at] = x;
  else
    static_cast<uint16_t*>(base)[at] = dt == kF16 ? narrow1<kF16>(x) : narrow1<kBF16>(x);
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
  return x + __builtin_bit_cast(
                 float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf,
                                                    true));
}
// The sum of the values of the lane's 16, 32 or 64, in a fixed order, in every lane.
// Every one of these must be active.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float x) {
  x = dpp_add<0xb1>(x);   // lanes xor 1
  x = dpp_add<0x4e>(x);   // xor 2
  x = dpp_add<0x141>(x);  // mirrored in eights
  x = dpp_add<0x140>(x);  // mirrored in sixteens
  const int b = __builtin_bit_cast(int, x);
  if constexpr (LANES == 16) return x;
  if constexpr (LANES == 32)
    return x + __builtin_bit_cast(float, __builtin_amdgcn_ds_swizzle(b, 0x401f));  // xor 16
  const float r0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 0));
  const float r1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 16));
  const float r2 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 32));
  const float r3 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 48));
  return (r0 + r1) + (r2 + r3);
}

}  // namespace
}  // namespace zs
