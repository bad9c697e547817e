// zs_adamw_step.h -- the AdamW step's kernel, compiled once per width of the
// moments (zs_adamw32.hip, zs_adamw8.hip).
#pragma once

#include "zs_adamw_device.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

// One block of 256 elements by one wave.  n < 0: a whole block; else the lane's
// n (0..4) elements of a tensor's last block.
template <int GDT, int PDT, int BITS, bool RANDOM, bool ONE>
__device__ __forceinline__ void step_block(const AwArgs& a, const AwConsts& c, const Chunk& ch,
                                           float GS, float LR, float LD, int b, uint32_t lane,
                                           int n) {
  const int64_t e = static_cast<int64_t>(b) * kStateBlock;
  float g[kQuad], w[kQuad], m[kQuad], v[kQuad];
  Raw4<kF32> mq, vq;
  uint32_t mc, vc;
  float ms, vs;
  Raw4<GDT> gq;
  if constexpr (ONE) {
    // a single gradient goes through plain loads beside 32-bit moments (1.0e9
    // elements 4.32 ms, 4.48 with non-temporal ones), non-temporal ones beside
    // 8-bit moments (2.63, plain 2.65) and from several ranks (15.6M elements,
    // 8 ranks 106 us, 111 with plain ones)
    const char* gb = ch.g + e * kSize<GDT>;
    gq = n < 0 ? ld_raw4<GDT, BITS == 8>(gb, lane) : ld_raw4<GDT>(gb, lane, n);
  }
  const Raw4<kF32> wq = n < 0 ? ld_raw4<kF32>(ch.w + e, lane) : ld_raw4<kF32>(ch.w + e, lane, n);
  if constexpr (BITS == 32) {
    const float* mb = reinterpret_cast<const float*>(ch.m) + e;
    const float* vb = reinterpret_cast<const float*>(ch.v) + e;
    mq = n < 0 ? ld_raw4<kF32>(mb, lane) : ld_raw4<kF32>(mb, lane, n);
    vq = n < 0 ? ld_raw4<kF32>(vb, lane) : ld_raw4<kF32>(vb, lane, n);
  } else {
    mc = n < 0 ? ld_codes(ch.m + e, lane) : ld_codes(ch.m + e, lane, n);
    vc = n < 0 ? ld_codes(ch.v + e, lane) : ld_codes(ch.v + e, lane, n);
    ms = ch.m_scale[b];
    vs = ch.v_scale[b];
  }
  if constexpr (ONE)
    widen4<GDT>(gq, g);
  else
    mean_ranks<GDT>(rank_ptrs(a.gptrs, ch.piece, a.p), a.p, a.PF, ch.start + e, lane, n, g);
  widen4<kF32>(wq, w);
  if constexpr (BITS == 32) {
    widen4<kF32>(mq, m);
    widen4<kF32>(vq, v);
  } else {
    decode4<ZS_STATE8_M>(mc, ms, m);
    decode4<ZS_STATE8_V>(vc, vs, v);
  }
#pragma unroll
  for (int j = 0; j < kQuad; ++j) {
    moments1(c, g[j] * GS, m[j], v[j]);
    float x;
    if constexpr (BITS == 32) {
      x = (m[j] / c.A1) / (__builtin_sqrtf(v[j] / c.A2) + c.EPS);
    } else {
      // the hardware's root and reciprocal: the 8-bit step is as much bound by
      // its arithmetic as by HBM, and moments that are held to 2^-4 need no
      // correctly rounded quotient
      x = m[j] * __builtin_amdgcn_rcpf(__builtin_amdgcn_sqrtf(v[j]) * c.R2 + c.EPS);
    }
    w[j] = w[j] - (LR * x + LD * w[j]);
  }
  if (n < 0) {
    st_quad32(ch.w + e, lane, w);
    if (ch.param) st_quad16<PDT>(ch.param + e, lane, w);
  } else {
    st_quad32(ch.w + e, lane, n, w);
    if (ch.param) st_quad16<PDT>(ch.param + e, lane, n, w);
  }
  if constexpr (BITS == 32) {
    float* mb = reinterpret_cast<float*>(ch.m) + e;
    float* vb = reinterpret_cast<float*>(ch.v) + e;
    if (n < 0) {
      st_quad32(mb, lane, m);
      st_quad32(vb, lane, v);
    } else {
      st_quad32(mb, lane, n, m);
      st_quad32(vb, lane, n, v);
    }
  } else {
    // elements behind the tensor's end are zeros here: they raise no maximum
    // (v is never negative, so its bits are its magnitude's)
    uint32_t mm = 0, vm = 0;
#pragma unroll
    for (int j = 0; j < kQuad; ++j) {
      mm = mag_bits(m[j]) > mm ? mag_bits(m[j]) : mm;
      vm = __float_as_uint(v[j]) > vm ? __float_as_uint(v[j]) : vm;
    }
    BlockScale sm, sv;
    float mine;
    block_scales(wave_max(mm), wave_max(vm), lane, sm, sv, mine);
    uint32_t word[kQuad] = {0u, 0u, 0u, 0u};
    if constexpr (RANDOM)
      philox(static_cast<uint64_t>(ch.index + e + kQuad * lane), static_cast<uint64_t>(c.step),
             a.seed, word);
    const uint32_t cm = encode4<ZS_STATE8_M, RANDOM>(m, sm, word);
    const uint32_t cv = encode4<ZS_STATE8_V, RANDOM>(v, sv, word);
    if (n < 0) {
      st_codes(ch.m + e, lane, cm);
      st_codes(ch.v + e, lane, cv);
    } else {
      st_codes(ch.m + e, lane, n, cm);
      st_codes(ch.v + e, lane, n, cv);
    }
    if (lane % (kWave / 2) == 0) (lane == 0 ? ch.m_scale : ch.v_scale)[b] = mine;
  }
}

// One block per wave, W waves per workgroup.  The grid sweeps the tensors in
// order, so what is in flight at any moment is a narrow window of each array;
// launch_step says which W keeps it narrowest.  (More blocks per wave were
// timed before W was chosen and the LDS below held waves back, 1.0e9 elements
// with 32-bit moments: 4.96 ms with one block, 5.12 with two, 5.35 with eight;
// and with 8-bit moments as they are now: 2.53, 2.91 with two, 2.98 with four.)
template <int W, int GDT, int PDT, int BITS, bool RANDOM, bool ONE>
__global__ __launch_bounds__(W * kWave) void adamw_kernel(AwArgs a) {
  const Chunk ch = ld_chunk(a.chunks + (blockIdx.x >> a.shift));
  const int wave = W == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int b = static_cast<int>(blockIdx.x & ((1u << a.shift) - 1u)) * W + wave;
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
    step_block<GDT, PDT, BITS, RANDOM, ONE>(a, c, ch, s.GS, LR, LD, b, lane, -1);
  } else {
    int n = left - kQuad * static_cast<int>(lane);
    n = n < 0 ? 0 : n > kQuad ? kQuad : n;
    step_block<GDT, PDT, BITS, RANDOM, ONE>(a, c, ch, s.GS, LR, LD, b, lane, n);
  }
}

// Waves per workgroup, and LDS that a 32-bit step asks for and leaves alone so
// that 16 waves share a CU instead of 32.  All figures with input sets that
// take turns, as a training step's do; 1.0e9 elements except where stated.
// 32-bit moments, one gradient: single waves, 16 of them: 4.27-4.38 ms (6.4-6.6
// TB/s); 12 / 14 / 20 / 24 / 32 per CU 4.78 / 4.61 / 4.43 / 4.54 / 4.68, two
// waves per workgroup 4.47-4.49, four 4.63, eight 4.77.
// 32-bit moments, several gradients: eight waves, two such workgroups on a CU:
// 15.6M elements and 8 ranks 105.6 us (four waves 107.6, sixteen 112); from
// kManyRanks on four waves, two such: 30M elements and 16 ranks 273 us against
// 292, 15M and 64 ranks 399 against 423.  Around the switch, 15M elements, eight
// / four waves: 8 ranks 103 / 111, 12 ranks 125 / 128, 14 ranks 137 / 149, 16
// ranks 143 / 142, 20 ranks 167 / 169, 24 ranks 185 / 185, 32 ranks 236 / 233.
// 8-bit moments, as many waves as fit (they compute more per byte): with one
// gradient two waves where all arrays begin on a line, 2.53 ms (four 2.56,
// eight 2.57-2.61), else eight, 2.80 (two 3.24, four 2.99); with several
// eight, 15.6M elements and 8 ranks in buffers that begin 3 elements into a line
// 85.0 us (four 88.3, two 92.2; on lines 74).  Of 64 ranks: 15M elements 380 us.
// A small table's chunks have four blocks, which is four waves at most.
constexpr unsigned kReserveOne = 160 * 1024 / 16 - 64, kReserveRanks = 160 * 1024 / 2 - 64;
constexpr int kManyRanks = 16;

template <int BITS, bool RANDOM>
void launch_step(const AwLaunch& L) {
  with_gdt(L.gdt, [&](auto G) {
    with_dt(L.pdt, [&](auto H) {
      constexpr int GDT = decltype(G)::value, PDT = decltype(H)::value;
      const auto go = [&](auto waves, auto one, unsigned lds) {
        constexpr int W = decltype(waves)::value;
        AwArgs a = L.a;
        a.shift = L.log_blocks - log2_of(W);
        adamw_kernel<W, GDT, PDT, BITS, RANDOM, decltype(one)::value != 0>
            <<<dim3(static_cast<unsigned>(L.nchunks << a.shift)), dim3(W * kWave), lds,
               L.stream>>>(a);
      };
      const bool small = L.log_blocks < log2_of(8);
      if constexpr (BITS == 32) {
        const unsigned lds = small ? 0 : kReserveRanks;
        if (L.a.p == 1)
          go(IC<1>{}, IC<1>{}, kReserveOne);
        else if (small || L.a.p >= kManyRanks)
          go(IC<4>{}, IC<0>{}, lds);
        else
          go(IC<8>{}, IC<0>{}, lds);
      } else if (L.a.p == 1) {
        if (L.on_lines)
          go(IC<2>{}, IC<1>{}, 0);
        else
          small ? go(IC<4>{}, IC<1>{}, 0) : go(IC<8>{}, IC<1>{}, 0);
      } else {
        small ? go(IC<4>{}, IC<0>{}, 0) : go(IC<8>{}, IC<0>{}, 0);
      }
    });
  });
}

}  // namespace
}  // namespace zs
