// zs_adamw.cpp -- host side of the AdamW operators: argument checks, the
// launch table, the step's constants.  Every argument error is returned before
// anything touches the device.

#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "zs_adamw.h"

namespace {

constexpr int64_t kMaxLen = int64_t{1} << 60;
using zs::kMaxGroups;

// Elements per entry of the launch table: 8192, or 1024 in tables of fewer than
// 512 such or of tensors that are shorter on average: short tensors then launch
// no idle waves (200,000 elements in 300 tensors, 32-bit moments 4.5 us, 9.1
// with 8192; their norm 4.9, 5.4).  Both sizes on both sides of the 512, which
// is 4.2M elements, 35 tensors, us with 1024 / 8192:
//   elements                     1.0e6        4.0e6        8.0e6      1.6e7
//   32 bits, one gradient     7.1 /  8.0  20.8 / 20.9  37.5 / 38.0   70 /  72
//   32 bits, 8 ranks         10.2 / 12.2  30.0 / 30.0  57.8 / 57.0  112 / 111
//   8 bits, 8 ranks          11.0 / 11.8  24.0 / 23.8  43.6 / 40.9   76 /  75
//   norm, one gradient        6.0 /  5.3   6.7 /  6.6   8.9 /  8.1   12 /  11
// (the norm of 1.0e6 is one launch with 1024 and two with 8192, which cost the
// host 2.4 us more).  1.0e9 elements, 32 bits, one gradient: 4.29 / 4.35 ms, in a
// table of eight times the bytes.
constexpr int kUnitsLarge = 3, kUnitsSmall = 0;
constexpr int64_t kChunkLarge = int64_t{zs::kUnit} << kUnitsLarge;
constexpr int64_t kChunkSmall = int64_t{zs::kUnit} << kUnitsSmall;

int64_t chunk_rule(int64_t total, int32_t npieces) {
  return total / kChunkLarge >= std::max(512, npieces) ? kChunkLarge : kChunkSmall;
}
int units_of(int64_t chunk) { return chunk == kChunkLarge ? kUnitsLarge : kUnitsSmall; }
// Blocks of 256 elements per entry, a power of two's exponent.
int log_blocks_of(int64_t chunk) {
  return units_of(chunk) + zs::log2_of(zs::kUnit / zs::kStateBlock);
}

// Where the workspace's parts lie: the entries, the rank pointers, the norm's
// count of arrivals and its partial sums (which alone are not uploaded).
struct Layout {
  size_t chunks, gptrs, arrived, partial, total;
};

size_t up256(size_t x) { return (x + 255u) & ~static_cast<size_t>(255u); }

Layout layout(int64_t nchunks, int32_t npieces, int32_t p) {
  Layout l;
  l.chunks = 0;
  l.gptrs = up256(sizeof(zs::AwChunk) * static_cast<size_t>(nchunks));
  l.arrived = l.gptrs + up256(sizeof(void*) * static_cast<size_t>(npieces) *
                              static_cast<size_t>(p));
  l.partial = l.arrived + 256;
  l.total = l.partial + up256(sizeof(double) * zs::kSumsqBlocks);
  return l;
}

// A tensor's first chunk may be up to kHeadMost - 1 elements short, so that the
// others begin on whole lines of memory (head_of).
constexpr int kHeadMost = 64;

// Chunks of a tensor whose first one is `head` short of a chunk or, with head
// 0, whole.
int64_t chunks_of(int64_t len, int64_t chunk, int head) {
  const int64_t first = head == 0 ? chunk : chunk - kHeadMost + head;
  return len <= first ? 1 : 1 + (len - first - 1) / chunk + 1;
}

// The most chunks that a list of tensors may come to, and the workspace for
// them; false if they are too many for a launch.
template <class Len>
bool plan(int32_t npieces, int32_t p, Len len, int64_t* chunk, int64_t* nchunks, Layout* out) {
  int64_t total = 0;
  for (int32_t i = 0; i < npieces; ++i) {
    if (len(i) < 1 || len(i) > kMaxLen || total > kMaxLen - len(i)) return false;
    total += len(i);
  }
  *chunk = chunk_rule(total, npieces);
  *nchunks = 0;
  for (int32_t i = 0; i < npieces; ++i) *nchunks += chunks_of(len(i), *chunk, 1);
  if (*nchunks > kMaxGroups >> units_of(*chunk)) return false;
  *out = layout(*nchunks, npieces, p);
  return true;
}

struct Span {
  uintptr_t lo, hi;
};

// An array of a tensor: where it begins, its element size, and the bytes per
// element that it moves.
struct Stream {
  uintptr_t at;
  unsigned size, weight;
};

// The elements (0..63) before the first chunk boundary of a tensor, chosen so
// that from there on its arrays' accesses start as near to whole 128-byte
// lines as they can.  1.0e9 elements with 32-bit moments in buffers that begin
// 12 bytes into a line: 6.09 ms with chunks from the first element on, 4.32
// with this (4.34 where all begin on a line); 30M, 3 ranks, 52 bytes into one:
// 173 us and 158.
int head_of(const std::vector<Stream>& streams) {
  int best = 0, best_score = -1;
  for (int h = 0; h < kHeadMost; ++h) {
    int score = 0;
    for (const Stream& s : streams) {
      const uintptr_t a = s.at + static_cast<uintptr_t>(h) * s.size;
      const int level = a % 128u == 0 ? 8 : a % 64u == 0 ? 6 : a % 16u == 0 ? 2 : a % 8u == 0;
      score += level * static_cast<int>(s.weight);
    }
    if (score > best_score) {
      best_score = score;
      best = h;
    }
  }
  return best;
}

bool grad_dtype_ok(int32_t dt) { return dt == ZS_F16 || dt == ZS_BF16 || dt == ZS_F32; }
bool param_dtype_ok(int32_t dt) { return dt == 0 || dt == ZS_F16 || dt == ZS_BF16; }

zs_status upload(const zs_adamw_piece* pieces, int32_t npieces, int32_t p, int32_t grad_dtype,
                 int32_t param_dtype, int32_t state_bits, void* workspace, size_t ws_bytes,
                 void* stream, zs_adamw_table* table) {
  if (!table || !workspace || (npieces > 0 && !pieces)) return ZS_ERR_NULL;
  if (p < 1 || p > ZS_MAX_P || npieces < 0 ||
      (state_bits != 0 && state_bits != 8 && state_bits != 32))
    return ZS_ERR_ARG;
  if (!grad_dtype_ok(grad_dtype) || !param_dtype_ok(param_dtype)) return ZS_ERR_DTYPE;
  const uintptr_t gsize = grad_dtype == ZS_F32 ? 4 : 2, ssize = state_bits == 8 ? 1 : 4;

  std::vector<Span> writes, reads;
  bool aligned = true;
  const auto span = [&](std::vector<Span>& to, const void* at, uintptr_t size, int64_t n) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(at);
    aligned = aligned && lo % size == 0;
    to.push_back({lo, lo + size * static_cast<uintptr_t>(n)});
  };
  bool all_mean = npieces > 0, on_lines = true;
  for (int32_t i = 0; i < npieces; ++i) {
    const zs_adamw_piece& q = pieces[i];
    if (q.len < 1 || q.len > kMaxLen || q.index < 0 || q.index > kMaxLen) return ZS_ERR_ARG;
    if (!q.grads) return ZS_ERR_NULL;
    for (int32_t r = 0; r < p; ++r) {
      if (!q.grads[r]) return ZS_ERR_NULL;
      span(reads, q.grads[r], gsize, q.len);
    }
    all_mean = all_mean && q.g_mean;
    if (q.g_mean) span(writes, q.g_mean, 4, q.len);
    if (state_bits == 0) continue;
    if (!std::isfinite(q.weight_decay) || q.weight_decay < 0.0 || !std::isfinite(q.lr_scale))
      return ZS_ERR_ARG;
    if (!q.w || !q.m || !q.v || (param_dtype != 0 && !q.param)) return ZS_ERR_NULL;
    span(writes, q.w, 4, q.len);
    span(writes, q.m, ssize, q.len);
    span(writes, q.v, ssize, q.len);
    if (param_dtype != 0) span(writes, q.param, 2, q.len);
    for (const void* at : {static_cast<const void*>(q.w), static_cast<const void*>(q.m),
                           static_cast<const void*>(q.v),
                           static_cast<const void*>(param_dtype != 0 ? q.param : nullptr)})
      on_lines = on_lines && reinterpret_cast<uintptr_t>(at) % 128 == 0;
    if (state_bits == 8) {
      if (!q.m_scale || !q.v_scale) return ZS_ERR_NULL;
      const int64_t nb = (q.len - 1) / ZS_STATE8_BLOCK + 1;
      span(writes, q.m_scale, 4, nb);
      span(writes, q.v_scale, 4, nb);
    }
  }
  if (!aligned) return ZS_ERR_ARG;

  Layout lay;
  int64_t chunk, nchunks;
  if (!plan(npieces, p, [&](int32_t i) { return pieces[i].len; }, &chunk, &nchunks, &lay))
    return ZS_ERR_RANGE;
  if (reinterpret_cast<uintptr_t>(workspace) % 256u != 0 || ws_bytes < lay.total)
    return ZS_ERR_CAPACITY;

  // Nothing written may meet anything else: sort, then sweep.
  const uintptr_t ws = reinterpret_cast<uintptr_t>(workspace);
  writes.push_back({ws, ws + lay.total});
  const auto by_lo = [](const Span& x, const Span& y) { return x.lo < y.lo; };
  std::sort(writes.begin(), writes.end(), by_lo);
  std::sort(reads.begin(), reads.end(), by_lo);
  for (size_t i = 1; i < writes.size(); ++i)
    if (writes[i].lo < writes[i - 1].hi) return ZS_ERR_ALIAS;
  size_t j = 0;
  uintptr_t reach = 0;  // the furthest end of a read that begins before this write's end
  for (const Span& wr : writes) {
    for (; j < reads.size() && reads[j].lo < wr.hi; ++j) reach = std::max(reach, reads[j].hi);
    if (reach > wr.lo) return ZS_ERR_ALIAS;
  }

  // Where the chunks begin.  Blocks of 8-bit moments are counted from their
  // tensor's first element, so there only the whole tensor can be aligned.
  std::vector<int> heads(static_cast<size_t>(npieces), 0);
  nchunks = 0;
  for (int32_t i = 0; i < npieces; ++i) {
    const zs_adamw_piece& q = pieces[i];
    if (state_bits != 8) {
      std::vector<Stream> streams;
      const auto add = [&](const void* at, unsigned size, unsigned weight) {
        if (at) streams.push_back({reinterpret_cast<uintptr_t>(at), size, weight});
      };
      for (int32_t r = 0; r < p; ++r)
        add(q.grads[r], static_cast<unsigned>(gsize), static_cast<unsigned>(gsize));
      if (state_bits == 32) {
        add(q.w, 4, 8);
        add(q.m, 4, 8);
        add(q.v, 4, 8);
        if (param_dtype != 0) add(q.param, 2, 2);
      }
      if (state_bits == 0) add(q.g_mean, 4, 4);
      heads[static_cast<size_t>(i)] = head_of(streams);
    }
    nchunks += chunks_of(q.len, chunk, heads[static_cast<size_t>(i)]);
  }
  lay = layout(nchunks, npieces, p);

  std::vector<unsigned char> host(lay.partial, 0);
  auto* chunks = reinterpret_cast<zs::AwChunk*>(host.data() + lay.chunks);
  auto* gptrs = reinterpret_cast<uint64_t*>(host.data() + lay.gptrs);
  const auto at = [](const void* p, uintptr_t size, int64_t n) {
    return p ? reinterpret_cast<uintptr_t>(p) + size * static_cast<uintptr_t>(n) : 0;
  };
  int64_t c = 0;
  for (int32_t i = 0; i < npieces; ++i) {
    const zs_adamw_piece& q = pieces[i];
    for (int32_t r = 0; r < p; ++r)
      gptrs[static_cast<int64_t>(i) * p + r] = at(q.grads[r], gsize, 0);
    const int head = heads[static_cast<size_t>(i)];
    int64_t n = head == 0 ? chunk : chunk - kHeadMost + head;
    for (int64_t e = 0; e < q.len; e += n, n = chunk) {
      n = std::min(n, q.len - e);
      zs::AwChunk& d = chunks[c++];
      if (state_bits != 0) {
        d.w = at(q.w, 4, e);
        d.m = at(q.m, ssize, e);
        d.v = at(q.v, ssize, e);
        if (state_bits == 8) {
          d.m_scale = at(q.m_scale, 4, e / ZS_STATE8_BLOCK);
          d.v_scale = at(q.v_scale, 4, e / ZS_STATE8_BLOCK);
        }
        if (param_dtype != 0) d.param = at(q.param, 2, e);
        d.lr_scale = q.lr_scale;
        d.decay = q.weight_decay;
      }
      d.g = at(q.grads[0], gsize, e);
      d.g_mean = at(q.g_mean, 4, e);
      d.index = q.index + e;
      d.start = e;
      d.len = static_cast<int32_t>(n);
      d.piece = i;
    }
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = hipMemcpyAsync(workspace, host.data(), host.size(), hipMemcpyHostToDevice, s);
  if (e == hipSuccess) e = hipStreamSynchronize(s);
  if (e != hipSuccess) return static_cast<zs_status>(zs::hip_status(e));
  table->workspace = workspace;
  table->nchunks = nchunks;
  table->chunk_elems = chunk;
  table->npieces = npieces;
  table->p = p;
  table->grad_dtype = grad_dtype;
  table->param_dtype = state_bits != 0 ? param_dtype : 0;
  table->state_bits = state_bits;
  table->has_mean = all_mean ? 1 : 0;
  table->on_lines = on_lines ? 1 : 0;
  table->reserved = 0;
  return ZS_OK;
}

zs_status check_table(const zs_adamw_table* t) {
  if (!t || !t->workspace) return ZS_ERR_NULL;
  if (t->p < 1 || t->p > ZS_MAX_P || t->npieces < 0 || t->nchunks < t->npieces ||
      (t->chunk_elems != kChunkLarge && t->chunk_elems != kChunkSmall) ||
      t->nchunks > kMaxGroups >> units_of(t->chunk_elems) ||
      (t->state_bits != 0 && t->state_bits != 8 && t->state_bits != 32))
    return ZS_ERR_ARG;
  if (!grad_dtype_ok(t->grad_dtype) || !param_dtype_ok(t->param_dtype)) return ZS_ERR_DTYPE;
  return ZS_OK;
}

zs_status check_hparams(const zs_adamw_hparams* h) {
  if (!h) return ZS_ERR_NULL;
  if (!std::isfinite(h->lr) || !std::isfinite(h->eps) || h->eps < 0.0) return ZS_ERR_ARG;
  if (!(h->beta1 >= 0.0 && h->beta1 < 1.0) || !(h->beta2 >= 0.0 && h->beta2 < 1.0))
    return ZS_ERR_ARG;
  if (h->step < 1 || !std::isfinite(h->grad_scale) || h->grad_scale == 0.0) return ZS_ERR_ARG;
  if (!std::isfinite(h->max_norm) || h->max_norm < 0.0) return ZS_ERR_ARG;
  if (h->rounding != ZS_ROUND_NEAREST && h->rounding != ZS_ROUND_STOCHASTIC) return ZS_ERR_ARG;
  if (h->skip_nonfinite != 0 && h->skip_nonfinite != 1) return ZS_ERR_ARG;
  return ZS_OK;
}

zs::AwConsts make_consts(const zs_adamw_hparams& h) {
  zs::AwConsts c;
  const double t = static_cast<double>(h.step);
  const double bc1 = 1.0 - std::pow(h.beta1, t), bc2 = 1.0 - std::pow(h.beta2, t);
  c.B1 = static_cast<float>(h.beta1);
  c.C1 = static_cast<float>(1.0 - h.beta1);
  c.B2 = static_cast<float>(h.beta2);
  c.C2 = static_cast<float>(1.0 - h.beta2);
  c.A1 = static_cast<float>(bc1);
  c.A2 = static_cast<float>(bc2);
  c.R2 = static_cast<float>(1.0 / std::sqrt(bc2));
  c.EPS = static_cast<float>(h.eps);
  c.inv_bc1 = 1.0 / bc1;
  c.lr = h.lr;
  c.step = h.step;
  return c;
}

zs_status from_hip(hipError_t e) {
  return e == hipSuccess ? ZS_OK : static_cast<zs_status>(zs::hip_status(e));
}

zs_status check_steps(const zs_adamw_steps* s) {
  if (!s || !s->dev) return ZS_ERR_NULL;
  if (s->nsteps < 1 || s->nsteps > ZS_MAX_TABLE_STEPS || s->reserved != 0) return ZS_ERR_ARG;
  return ZS_OK;
}

zs_status adamw_step(const zs_adamw_table* t, const zs_adamw_steps* steps,
                     const zs_adamw_hparams* hp, const double* sumsq, void* stream) {
  if (const zs_status st = check_table(t)) return st;
  if (const zs_status st = check_hparams(hp)) return st;
  if (t->state_bits == 0) return ZS_ERR_ARG;
  if (!sumsq && (hp->max_norm > 0.0 || hp->skip_nonfinite)) return ZS_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(sumsq) % sizeof(double) != 0) return ZS_ERR_ARG;
  if (t->nchunks == 0) return ZS_OK;
  const Layout lay = layout(t->nchunks, t->npieces, t->p);
  auto* base = static_cast<unsigned char*>(t->workspace);
  zs::AwLaunch L;
  L.a.chunks = reinterpret_cast<const zs::AwChunk*>(base + lay.chunks);
  L.a.gptrs = reinterpret_cast<const uint64_t*>(base + lay.gptrs);
  L.a.sumsq = sumsq;
  L.a.steps = steps ? static_cast<zs::AwStepsDev*>(steps->dev) : nullptr;
  L.a.grad_scale = hp->grad_scale;
  L.a.max_norm = hp->max_norm;
  L.a.seed = hp->seed;
  L.a.p = t->p;
  L.a.skip_nonfinite = hp->skip_nonfinite;
  L.log_blocks = log_blocks_of(t->chunk_elems);
  L.a.PF = static_cast<float>(static_cast<double>(t->p));
  L.a.c = make_consts(*hp);
  L.nchunks = t->nchunks;
  L.gdt = t->grad_dtype;
  L.pdt = t->param_dtype ? t->param_dtype : ZS_BF16;
  L.rounding = hp->rounding;
  L.on_lines = t->on_lines != 0;
  L.stream = static_cast<hipStream_t>(stream);
  return from_hip(t->state_bits == 32 ? zs::launch_adamw32(L) : zs::launch_adamw8(L));
}

size_t steps_bytes(int32_t nsteps) {
  if (nsteps < 1 || nsteps > ZS_MAX_TABLE_STEPS) return 0;
  return up256(sizeof(zs::AwStepsDev) + sizeof(zs::AwConsts) * static_cast<size_t>(nsteps));
}

zs_status steps_init(const zs_adamw_hparams* hp, const double* lrs, int32_t nsteps, void* dev,
                     size_t bytes, void* stream, zs_adamw_steps* out) {
  if (!out || !dev) return ZS_ERR_NULL;
  if (const zs_status st = check_hparams(hp)) return st;
  if (nsteps < 1 || nsteps > ZS_MAX_TABLE_STEPS) return ZS_ERR_ARG;
  if (hp->step > INT64_MAX - nsteps) return ZS_ERR_RANGE;
  for (int32_t i = 0; lrs && i < nsteps; ++i)
    if (!std::isfinite(lrs[i])) return ZS_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(dev) % 256u != 0 || bytes < steps_bytes(nsteps))
    return ZS_ERR_CAPACITY;
  std::vector<unsigned char> host(steps_bytes(nsteps), 0);
  reinterpret_cast<zs::AwStepsDev*>(host.data())->nsteps = nsteps;
  auto* entry = reinterpret_cast<zs::AwConsts*>(host.data() + sizeof(zs::AwStepsDev));
  zs_adamw_hparams h = *hp;
  for (int32_t i = 0; i < nsteps; ++i) {
    h.step = hp->step + i;
    if (lrs) h.lr = lrs[i];
    entry[i] = make_consts(h);
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = hipMemcpyAsync(dev, host.data(), host.size(), hipMemcpyHostToDevice, s);
  if (e == hipSuccess) e = hipStreamSynchronize(s);
  if (e != hipSuccess) return from_hip(e);
  out->dev = dev;
  out->first_step = hp->step;
  out->nsteps = nsteps;
  out->reserved = 0;
  return ZS_OK;
}

zs_status convert_args(const float* x, const void* codes, const float* scales, int64_t n,
                       int32_t kind) {
  if (kind != ZS_STATE8_M && kind != ZS_STATE8_V) return ZS_ERR_ARG;
  if (n < 0) return ZS_ERR_ARG;
  if (n > kMaxLen) return ZS_ERR_RANGE;
  if (n == 0) return ZS_OK;
  if (!x || !codes || !scales) return ZS_ERR_NULL;
  const uintptr_t px = reinterpret_cast<uintptr_t>(x), pc = reinterpret_cast<uintptr_t>(codes),
                  ps = reinterpret_cast<uintptr_t>(scales), u = static_cast<uintptr_t>(n);
  if (px % 4 != 0 || ps % 4 != 0) return ZS_ERR_ARG;
  const Span s[3] = {{px, px + 4 * u},
                     {pc, pc + u},
                     {ps, ps + 4 * ((u - 1) / ZS_STATE8_BLOCK + 1)}};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (s[i].lo < s[j].hi && s[j].lo < s[i].hi) return ZS_ERR_ALIAS;
  return ZS_OK;
}

}  // namespace

extern "C" {

size_t zs_adamw_workspace_bytes(const int64_t* lens, int32_t npieces, int32_t p) {
  if (npieces < 0 || (npieces > 0 && !lens) || p < 1 || p > ZS_MAX_P) return 0;
  Layout lay;
  int64_t chunk, nchunks;
  if (!plan(npieces, p, [&](int32_t i) { return lens[i]; }, &chunk, &nchunks, &lay)) return 0;
  return lay.total;
}

zs_status zs_adamw_upload(const zs_adamw_piece* pieces, int32_t npieces, int32_t p,
                          int32_t grad_dtype, int32_t param_dtype, int32_t state_bits,
                          void* workspace, size_t ws_bytes, void* stream, zs_adamw_table* table) {
  return zs::guard([&] {
    return upload(pieces, npieces, p, grad_dtype, param_dtype, state_bits, workspace, ws_bytes,
                  stream, table);
  });
}

zs_status zs_adamw_step_multi(const zs_adamw_table* table, const zs_adamw_hparams* hp,
                              const double* sumsq, void* stream) {
  return zs::guard([&] { return adamw_step(table, nullptr, hp, sumsq, stream); });
}

zs_status zs_adamw_step_multi_dev(const zs_adamw_table* table, const zs_adamw_steps* steps,
                                  const zs_adamw_hparams* hp, const double* sumsq, void* stream) {
  return zs::guard([&]() -> zs_status {
    if (const zs_status st = check_steps(steps)) return st;
    return adamw_step(table, steps, hp, sumsq, stream);
  });
}

size_t zs_adamw_steps_bytes(int32_t nsteps) { return steps_bytes(nsteps); }

zs_status zs_adamw_steps_init(const zs_adamw_hparams* hp, const double* lrs, int32_t nsteps,
                              void* dev, size_t bytes, void* stream, zs_adamw_steps* steps) {
  return zs::guard([&] { return steps_init(hp, lrs, nsteps, dev, bytes, stream, steps); });
}

zs_status zs_adamw_steps_advance(const zs_adamw_steps* steps, const double* sumsq, void* stream) {
  if (const zs_status st = check_steps(steps)) return st;
  if (reinterpret_cast<uintptr_t>(sumsq) % sizeof(double) != 0) return ZS_ERR_ARG;
  return from_hip(zs::launch_steps_advance(static_cast<zs::AwStepsDev*>(steps->dev), sumsq,
                                           static_cast<hipStream_t>(stream)));
}

zs_status zs_adamw_steps_status(const zs_adamw_steps* steps, int64_t* cursor, int32_t* exhausted,
                                void* stream) {
  if (const zs_status st = check_steps(steps)) return st;
  zs::AwStepsDev t;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = hipMemcpyAsync(&t, steps->dev, sizeof(t), hipMemcpyDeviceToHost, s);
  if (e == hipSuccess) e = hipStreamSynchronize(s);
  if (e != hipSuccess) return from_hip(e);
  if (cursor) *cursor = t.cursor;
  if (exhausted) *exhausted = t.exhausted;
  return ZS_OK;
}

zs_status zs_grad_sumsq_multi(const zs_adamw_table* t, int32_t store_mean, int32_t accumulate,
                              double* sumsq, void* stream) {
  return zs::guard([&]() -> zs_status {
    if (const zs_status st = check_table(t)) return st;
    if (!sumsq) return ZS_ERR_NULL;
    if ((store_mean != 0 && store_mean != 1) || (accumulate != 0 && accumulate != 1) ||
        reinterpret_cast<uintptr_t>(sumsq) % sizeof(double) != 0)
      return ZS_ERR_ARG;
    if (store_mean && t->npieces > 0 && !t->has_mean) return ZS_ERR_NULL;
    const Layout lay = layout(t->nchunks, t->npieces, t->p);
    auto* base = static_cast<unsigned char*>(t->workspace);
    const uintptr_t at = reinterpret_cast<uintptr_t>(sumsq), ws = reinterpret_cast<uintptr_t>(base);
    if (at < ws + lay.total && ws < at + sizeof(double)) return ZS_ERR_ALIAS;
    zs::SumsqLaunch L;
    L.chunks = reinterpret_cast<const zs::AwChunk*>(base + lay.chunks);
    L.gptrs = reinterpret_cast<const uint64_t*>(base + lay.gptrs);
    L.nchunks = t->nchunks;
    L.log_blocks = log_blocks_of(t->chunk_elems);
    L.p = t->p;
    L.gdt = t->grad_dtype;
    L.store = store_mean != 0;
    L.accumulate = accumulate != 0;
    L.partial = reinterpret_cast<double*>(base + lay.partial);
    L.arrived = reinterpret_cast<unsigned int*>(base + lay.arrived);
    L.out = sumsq;
    L.stream = static_cast<hipStream_t>(stream);
    return from_hip(zs::launch_sumsq(L));
  });
}

zs_status zs_state8_encode(const float* x, int64_t n, int32_t kind, void* codes, float* scales,
                           void* stream) {
  if (const zs_status st = convert_args(x, codes, scales, n, kind)) return st;
  if (n == 0) return ZS_OK;
  return from_hip(zs::launch_state8_encode(x, n, kind, codes, scales, static_cast<hipStream_t>(stream)));
}

zs_status zs_state8_decode(const void* codes, const float* scales, int64_t n, int32_t kind,
                           float* x, void* stream) {
  if (const zs_status st = convert_args(x, codes, scales, n, kind)) return st;
  if (n == 0) return ZS_OK;
  return from_hip(zs::launch_state8_decode(codes, scales, n, kind, x, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
