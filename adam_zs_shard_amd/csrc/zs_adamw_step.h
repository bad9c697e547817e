// zs_adamw_step.h -- the AdamW step's kernel, compiled once per width of the
// moments (zs_adamw32.hip, zs_adamw8.hip).
#pragma once

#include "zs_adamw_device.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

// U blocks of 256 elements by one wave, from block b of the chunk on.  n < 0:
// whole blocks; else (U = 1) the lane's n (0..4) elements of a tensor's last
// block.
template <int U, int GDT, int PDT, int BITS, bool RANDOM, bool ONE>
__device__ __forceinline__ void step_blocks(const AwArgs& a, const AwConsts& c, const Chunk& ch,
                                            float GS, float LR,
                                            float LD, int b, uint32_t lane, int n) {
  const int64_t e0 = static_cast<int64_t>(b) * kStateBlock;
  float g[U][kQuad], w[U][kQuad], m[U][kQuad], v[U][kQuad];
  Raw4<kF32> wq[U], mq[U], vq[U];
  uint32_t mc[U], vc[U];
  float ms[U], vs[U];
  Raw4<GDT> gq[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t e = e0 + u * kStateBlock;
    if constexpr (ONE) {
      // a single gradient goes through plain loads beside 32-bit moments (1.0e9
      // elements 4.79 -> 4.63 ms), non-temporal ones beside 8-bit moments
      // (equal) and from several ranks (15.6M elements, 8 ranks 107.5 us, 110.2
      // with plain ones)
      const char* gb = ch.g + e * kSize<GDT>;
      gq[u] = n < 0 ? ld_raw4<GDT, BITS == 8>(gb, lane) : ld_raw4<GDT>(gb, lane, n);
    }
    wq[u] = n < 0 ? ld_raw4<kF32>(ch.w + e, lane) : ld_raw4<kF32>(ch.w + e, lane, n);
    if constexpr (BITS == 32) {
      const float* mb = reinterpret_cast<const float*>(ch.m) + e;
      const float* vb = reinterpret_cast<const float*>(ch.v) + e;
      mq[u] = n < 0 ? ld_raw4<kF32>(mb, lane) : ld_raw4<kF32>(mb, lane, n);
      vq[u] = n < 0 ? ld_raw4<kF32>(vb, lane) : ld_raw4<kF32>(vb, lane, n);
    } else {
      mc[u] = n < 0 ? ld_codes(ch.m + e, lane) : ld_codes(ch.m + e, lane, n);
      vc[u] = n < 0 ? ld_codes(ch.v + e, lane) : ld_codes(ch.v + e, lane, n);
      ms[u] = ch.m_scale[b + u];
      vs[u] = ch.v_scale[b + u];
    }
  }
  if constexpr (ONE) {
#pragma unroll
    for (int u = 0; u < U; ++u) widen4<GDT>(gq[u], g[u]);
  } else {
    mean_ranks<U, GDT>(rank_ptrs(a.gptrs, ch.piece, a.p), a.p, a.PF, ch.start + e0, lane, n, g);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t e = e0 + u * kStateBlock;
    widen4<kF32>(wq[u], w[u]);
    if constexpr (BITS == 32) {
      widen4<kF32>(mq[u], m[u]);
      widen4<kF32>(vq[u], v[u]);
    } else {
      decode4<ZS_STATE8_M>(mc[u], ms[u], m[u]);
      decode4<ZS_STATE8_V>(vc[u], vs[u], v[u]);
    }
#pragma unroll
    for (int j = 0; j < kQuad; ++j) {
      moments1(c, g[u][j] * GS, m[u][j], v[u][j]);
      float x;
      if constexpr (BITS == 32) {
        x = (m[u][j] / c.A1) / (__builtin_sqrtf(v[u][j] / c.A2) + c.EPS);
      } else {
        // the hardware's root and reciprocal: the 8-bit step is as much bound
        // by its arithmetic as by HBM, and moments that are held to 2^-4 need
        // no correctly rounded quotient
        x = m[u][j] *
            __builtin_amdgcn_rcpf(__builtin_amdgcn_sqrtf(v[u][j]) * c.R2 + c.EPS);
      }
      w[u][j] = w[u][j] - (LR * x + LD * w[u][j]);
    }
    if (n < 0) {
      st_quad32(ch.w + e, lane, w[u]);
      if (ch.param) st_quad16<PDT>(ch.param + e, lane, w[u]);
    } else {
      st_quad32(ch.w + e, lane, n, w[u]);
      if (ch.param) st_quad16<PDT>(ch.param + e, lane, n, w[u]);
    }
    if constexpr (BITS == 32) {
      float* mb = reinterpret_cast<float*>(ch.m) + e;
      float* vb = reinterpret_cast<float*>(ch.v) + e;
      if (n < 0) {
        st_quad32(mb, lane, m[u]);
        st_quad32(vb, lane, v[u]);
      } else {
        st_quad32(mb, lane, n, m[u]);
        st_quad32(vb, lane, n, v[u]);
      }
    } else {
      // elements behind the tensor's end are zeros here: they raise no maximum
      // (v is never negative, so its bits are its magnitude's)
      uint32_t mm = 0, vm = 0;
#pragma unroll
      for (int j = 0; j < kQuad; ++j) {
        mm = mag_bits(m[u][j]) > mm ? mag_bits(m[u][j]) : mm;
        vm = __float_as_uint(v[u][j]) > vm ? __float_as_uint(v[u][j]) : vm;
      }
      BlockScale sm, sv;
      float mine;
      block_scales(wave_max(mm), wave_max(vm), lane, sm, sv, mine);
      uint32_t word[kQuad] = {0u, 0u, 0u, 0u};
      if constexpr (RANDOM)
        philox(static_cast<uint64_t>(ch.index + e + kQuad * lane),
               static_cast<uint64_t>(c.step), a.seed, word);
      const uint32_t cm = encode4<ZS_STATE8_M, RANDOM>(m[u], sm, word);
      const uint32_t cv = encode4<ZS_STATE8_V, RANDOM>(v[u], sv, word);
      if (n < 0) {
        st_codes(ch.m + e, lane, cm);
        st_codes(ch.v + e, lane, cv);
      } else {
        st_codes(ch.m + e, lane, n, cm);
        st_codes(ch.v + e, lane, n, cv);
      }
      if (lane % (kWave / 2) == 0) (lane == 0 ? ch.m_scale : ch.v_scale)[b + u] = mine;
    }
  }
}

// One workgroup per kUnit elements, one block per wave.  The grid sweeps the
// tensors in order, so what is in flight at any moment is a narrow window of
// each array: 1.0e9 elements with 32-bit moments take 4.96 ms this way, 5.12
// with 2048 elements per workgroup, 5.35 with 8192.
template <int GDT, int PDT, int BITS, bool RANDOM, bool ONE>
__global__ __launch_bounds__(kBlock) void adamw_kernel(AwArgs a) {
  const Chunk ch = ld_chunk(a.chunks + (blockIdx.x >> a.units));
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int b = static_cast<int>(blockIdx.x & ((1u << a.units) - 1u)) * kWaves + wave;
  const int left = ch.len - b * kStateBlock;
  if (left <= 0) return;
  const Scalars s = scalars(a);
  if (s.skip) return;
  AwConsts c = a.c;
  if (a.steps) {
    const int64_t at = a.steps->cursor;
    if (at < 0 || at >= a.steps->nsteps) {
      if (blockIdx.x == 0 && threadIdx.x == 0) a.steps->exhausted = 1;
      return;
    }
    c = reinterpret_cast<const AwConsts*>(a.steps + 1)[at];
  }
  const double lr = c.lr * ch.lr_scale;
  const float LR = static_cast<float>(BITS == 32 ? lr : lr * c.inv_bc1);
  const float LD = static_cast<float>(lr * ch.decay);
  const uint32_t lane = threadIdx.x % kWave;
  if (left >= kStateBlock) {
    step_blocks<1, GDT, PDT, BITS, RANDOM, ONE>(a, c, ch, s.GS, LR, LD, b, lane, -1);
  } else {
    int n = left - kQuad * static_cast<int>(lane);
    n = n < 0 ? 0 : n > kQuad ? kQuad : n;
    step_blocks<1, GDT, PDT, BITS, RANDOM, ONE>(a, c, ch, s.GS, LR, LD, b, lane, n);
  }
}

// LDS that the 32-bit step asks for and leaves alone: a fifth of a CU's 160
// KiB, so that five workgroups share a CU instead of eight.  Fewer waves in
// flight keep the sweep's window on HBM narrower: 1.0e9 elements 4.93 ms
// without, 4.77 / 4.76 / 4.75 / 4.85 with four, five, six and seven; 20M
// elements 91.5 -> 89.4 us.  The 8-bit step, which computes more per byte,
// needs the waves (2.63 ms with eight, 2.98 with five).
constexpr unsigned kReserve = 160 * 1024 / 5 - 64;

template <int BITS, bool RANDOM>
void launch_step(const AwLaunch& L) {
  with_gdt(L.gdt, [&](auto G) {
    with_dt(L.pdt, [&](auto H) {
      constexpr int GDT = decltype(G)::value, PDT = decltype(H)::value;
      const dim3 grid(static_cast<unsigned>(L.nchunks << L.a.units)), block(kBlock);
      constexpr unsigned lds = BITS == 32 ? kReserve : 0;
      if (L.a.p == 1)
        adamw_kernel<GDT, PDT, BITS, RANDOM, true><<<grid, block, lds, L.stream>>>(L.a);
      else
        adamw_kernel<GDT, PDT, BITS, RANDOM, false><<<grid, block, lds, L.stream>>>(L.a);
    });
  });
}

}  // namespace
}  // namespace zs
