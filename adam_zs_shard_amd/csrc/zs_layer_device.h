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

template <int V>
struct Vals {
  float v[V];
};

// The pack at `at`, or its first n elements and zeros behind them.
// Non-temporal unless STREAM is false.
template <int DT, bool STREAM = true>
__device__ __forceinline__ Pack<DT> ld_pack(const char* at) {
  const auto* p = reinterpret_cast<const decltype(Pack<DT>::x)*>(at);
  return Pack<DT>{STREAM ? __builtin_nontemporal_load(p) : *p};
}
template <int DT>
__device__ __forceinline__ Pack<DT> ld_part(const char* at, int n) {
  Pack<DT> q{};
  if constexpr (DT == kF32) {
#pragma unroll
    for (int i = 0; i < kPack<DT>; ++i)
      if (i < n) q.x[i] = reinterpret_cast<const float*>(at)[i];
  } else {
#pragma unroll
    for (int i = 0; i < kPack<DT>; ++i)
      if (i < n)
        q.x[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(at)[i]) << (16 * (i % 2));
  }
  return q;
}
// n >= kPack: the whole pack; n <= 0: zeros, nothing read.  WHOLE: one of the two.
template <int DT, bool WHOLE = false, bool STREAM = true>
__device__ __forceinline__ Pack<DT> ld_some(const char* at, int n) {
  if (n >= kPack<DT>) return ld_pack<DT, STREAM>(at);
  return !WHOLE && n > 0 ? ld_part<DT>(at, n) : Pack<DT>{};
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

template <int DT, bool WHOLE = false>
__device__ __forceinline__ void st_some(char* at, int n, const Pack<DT>& q) {
  if (n >= kPack<DT>) {
    __builtin_nontemporal_store(q.x, reinterpret_cast<decltype(Pack<DT>::x)*>(at));
  } else if (!WHOLE && n > 0) {
#pragma unroll
    for (int i = 0; i < kPack<DT>; ++i)
      if (i < n) {
        if constexpr (DT == kF32)
          reinterpret_cast<float*>(at)[i] = q.x[i];
        else
          reinterpret_cast<uint16_t*>(at)[i] = static_cast<uint16_t>(q.x[i / 2] >> (16 * (i % 2)));
      }
  }
}

// V elements at `at`, n of them there (the rest: `none`).
template <int V, int WDT>
__device__ __forceinline__ Vals<V> ld_vals(const char* at, int n, float none) {
  Vals<V> r;
  if (n >= V) {
    if constexpr (WDT == kF32) {
#pragma unroll
      for (int k = 0; k < V / 4; ++k) {
        const Pack<kF32> q = ld_pack<kF32, false>(at + 16 * k);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.v[4 * k + i] = q.x[i];
      }
    } else {
#pragma unroll
      for (int k = 0; k < V / 4; ++k) {
        const u32x2 q = reinterpret_cast<const u32x2*>(at)[k];
        r.v[4 * k] = widen_lo<WDT>(q[0]);
        r.v[4 * k + 1] = widen_hi<WDT>(q[0]);
        r.v[4 * k + 2] = widen_lo<WDT>(q[1]);
        r.v[4 * k + 3] = widen_hi<WDT>(q[1]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float x = none;
      if (i < n) {
        if constexpr (WDT == kF32)
          x = reinterpret_cast<const float*>(at)[i];
        else
          x = widen1<WDT>(reinterpret_cast<const uint16_t*>(at)[i]);
      }
      r.v[i] = x;
    }
  }
  return r;
}
// Rounds V values to `at`, n of them there.
template <int V, int DT>
__device__ __forceinline__ void st_vals(char* at, int n, const Vals<V>& x) {
  if constexpr (DT == kF32) {
#pragma unroll
    for (int k = 0; k < V / 4; ++k) {
      const float f[4] = {x.v[4 * k], x.v[4 * k + 1], x.v[4 * k + 2], x.v[4 * k + 3]};
      st_some<kF32>(at + 16 * k, n - 4 * k, narrow<kF32>(f));
    }
  } else if constexpr (V == 8) {
    st_some<DT>(at, n, narrow<DT>(x.v));
  } else {
    const u32x2 q{narrow_pair<DT>(x.v[0], x.v[1]), narrow_pair<DT>(x.v[2], x.v[3])};
    if (n >= 4) {
      __builtin_nontemporal_store(q, reinterpret_cast<u32x2*>(at));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) reinterpret_cast<uint16_t*>(at)[i] = static_cast<uint16_t>(q[i / 2] >> (16 * (i % 2)));
    }
  }
}
// Of a vector of weights, from element c on; no vector: `none`.
template <int V>
__device__ __forceinline__ Vals<V> ld_weights(const void* base, int wdt, int64_t c, int n, float none) {
  Vals<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.v[i] = none;
  if (base && n > 0) {
    const char* at = static_cast<const char*>(base) + c * (wdt == kF32 ? 4 : 2);
    if (wdt == kF16) r = ld_vals<V, kF16>(at, n, none);
    else if (wdt == kBF16) r = ld_vals<V, kBF16>(at, n, none);
    else r = ld_vals<V, kF32>(at, n, none);
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
// The sum of the wave's values, in a fixed order, in every lane.  Every lane
// must be active.
__device__ __forceinline__ float wave_sum(float x) {
  x = dpp_add<0xb1>(x);   // lanes xor 1
  x = dpp_add<0x4e>(x);   // xor 2
  x = dpp_add<0x141>(x);  // mirrored in eights
  x = dpp_add<0x140>(x);  // mirrored in sixteens
  const int b = __builtin_bit_cast(int, x);
  const float r0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 0));
  const float r1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 16));
  const float r2 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 32));
  const float r3 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 48));
  return (r0 + r1) + (r2 + r3);
}

}  // namespace
}  // namespace zs
