// Losses over packed sequences of tokens, from the tokens' losses nll = -log p
// that the vocabulary loss leaves, and their gradients by nll, which are the
// dloss that its backward takes.
//
// Policy loss, a value a sequence s:
//   d = old_nll - nll, r = e^d, A the advantage (of s, or of the token)
//   token = -min(r A, clip(r, 1 - lo, 1 + hi) A) + w k
//   k = e^x - 1 - x, x = nll - ref_nll
//   loss_s = sum over the tokens that count (/ their number N_s)
//   dnll = dloss_s (/ N_s) ([not clipped] r A + w (e^x - 1))
// Preference loss, a value a pair (sequences 2 i, preferred, and 2 i + 1):
//   reward_s = beta sum (ref_nll - nll) (/ N_s)
//   x_i = reward_2i - reward_2i+1 - margin,  loss_i = f(x_i)
//   dnll = -+ beta (/ N_s) dloss_i f'(x_i)
//
// Sequences are offsets in device memory, so no launch depends on their
// lengths: the tokens are cut into equal spans, a wave each, whatever
// sequences they belong to.  A wave walks its span in tiles of 512 tokens,
// eight to a lane, and finds the sequences that start in a tile from the
// offsets (a 64-way search once, then 64 offsets at a time).  Sums are fp64
// (the terms of a sequence cancel, and there may be millions): per lane where
// no sequence starts in a tile, else a segmented scan over the wave.  A
// sequence's part in the span where it starts goes to head[s], a span's part
// of the sequence that it starts within to carry[span], and a second kernel
// joins head[s] and the carries behind it in order: no atomics, the same bits
// every time.
#include <algorithm>
#include <cmath>

#include "train_common.h"

namespace muon {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kPer = 8, kTile = 64 * kPer;  // tokens of a lane, of a wave's tile

// first + 1 offsets, non-decreasing; whatever they hold, values are within
// [0, n].
struct Offsets {
  const int32_t* p;
  int count, n;  // sequences, tokens
  __device__ __forceinline__ int at(int s) const { return min(max(p[s], 0), n); }
};

// The sequences of a lane's eight tokens, tile by tile.
struct Walk {
  int next;  // the first sequence (count: the end) that starts at the tile or later

  // 64-way search: the number of offsets below `token`
  __device__ __forceinline__ void find(const Offsets& off, int token, int lane) {
    int lo = 0, len = off.count + 1;
    while (len > 0) {
      const int step = (len + 63) >> 6, q = lane * step + step - 1;
      const bool below = q < len && off.at(lo + q) < token;
      const int c = __popcll(__ballot(below));
      lo += c * step;
      len = min(step - 1, len - c * step);
    }
    next = __builtin_amdgcn_readfirstlane(lo);
  }
  // Marks the starts in the tile: start[j] is the sequence that starts at the
  // lane's token j, or -1; before: the one its first token is in unless it
  // starts there (-1 and count: none).  Returns whether any starts.
  __device__ __forceinline__ bool tile(const Offsets& off, int tile0, int lane, int* lds,
                                       int (&start)[kPer], int& before) {
    before = next - 1;
    bool any = false;
    for (;;) {
      const int s = next + lane;
      const int o = s <= off.count ? off.at(s) - tile0 : kTile;
      const uint64_t in = __ballot(o < kTile);
      if (in == 0) break;
      if (!any) {
        any = true;
#pragma unroll
        for (int j = 0; j < kPer; ++j) lds[lane * kPer + j] = -1;
        wave_sync();
      }
      // of several that start at a token all but the last are empty
      if (o >= 0 && o < kTile) atomicMax(&lds[o], s);
      const int c = __popcll(in);
      next += c;
      if (c < 64) break;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) start[j] = -1;
    if (!any) return false;
    wave_sync();
    int last = -1;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      start[j] = lds[lane * kPer + j];
      last = max(last, start[j]);
    }
    wave_sync();  // read before the next tile's marks
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(last, o, 64);
      if (lane >= o) last = max(last, u);
    }
    const int u = __shfl_up(last, 1, 64);
    if (lane > 0) before = max(before, u);
    return true;
  }
};

// Eight values from token i on, those below n; 0 past it.
template <typename T>
__device__ __forceinline__ void load_tokens(const T* p, int64_t i, int64_t n, T (&v)[kPer]) {
  if (i + kPer <= n) {
    __builtin_memcpy(v, p + i, sizeof(v));
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] = i + j < n ? p[i + j] : T{};
  }
}

// Sums over tokens.
struct Sums {
  double a, b;
  int c, d;
  __device__ __forceinline__ void add(const Sums& o) {
    a += o.a;
    b += o.b;
    c += o.c;
    d += o.d;
  }
  __device__ __forceinline__ Sums up(int o) const {
    return {__shfl_up(a, o, 64), __shfl_up(b, o, 64), __shfl_up(c, o, 64), __shfl_up(d, o, 64)};
  }
  __device__ __forceinline__ Sums other(int o) const {
    return {__shfl_xor(a, o, 64), __shfl_xor(b, o, 64), __shfl_xor(c, o, 64), __shfl_xor(d, o, 64)};
  }
  template <int G>
  __device__ __forceinline__ void join() {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) add(other(o));
  }
};

// e^x - 1 and e^x - 1 - x, whose difference of near values a polynomial
// replaces below |x| = 1/2: x^2 (1/2 + x / 6 + ... + x^6 / 40320), off by
// 2 x^7 / 9! < 2^-24 of itself.
__device__ __forceinline__ void exp_terms(float x, float& em1, float& k) {
  if (fabsf(x) < 0.5f) {
    float p = 1.0f / 40320.0f;
    p = __builtin_fmaf(p, x, 1.0f / 5040.0f);
    p = __builtin_fmaf(p, x, 1.0f / 720.0f);
    p = __builtin_fmaf(p, x, 1.0f / 120.0f);
    p = __builtin_fmaf(p, x, 1.0f / 24.0f);
    p = __builtin_fmaf(p, x, 1.0f / 6.0f);
    p = __builtin_fmaf(p, x, 0.5f);
    k = x * x * p;
    em1 = x + k;
  } else {
    em1 = expf(x) - 1.0f;
    k = em1 - x;
  }
}

struct PolicyArgs {
  const float *nll, *old_nll, *ref, *adv;
  const uint8_t* mask;
  // The clip as bounds of d: r > 1 + hi where d > log(1 + hi).  Compared in
  // fp64, where the difference of two fp32 values is exact but for the last bits
  // of very unlike ones: a ratio next to the border is on its own side of it.
  double d_low, d_high;
  float r_low, r_high, kl_weight;
  int per_token;

  __device__ __forceinline__ bool clipped(float a, double d) const {
    return (a > 0.0f && d > d_high) || (a < 0.0f && d < d_low);
  }
  // r A; no 0 inf where an advantage of 0 meets a ratio beyond fp32
  static __device__ __forceinline__ float ratio(float a, double d) {
    return a == 0.0f ? 0.0f : expf(static_cast<float>(d)) * a;
  }
};

struct PolicyTerms {
  PolicyArgs p;
  float nll[kPer], old_nll[kPer], ref[kPer], adv[kPer];
  uint8_t mask[kPer];
  __device__ __forceinline__ void load(int64_t i, int64_t n) {
    load_tokens(p.nll, i, n, nll);
    load_tokens(p.old_nll, i, n, old_nll);
    if (p.ref != nullptr) load_tokens(p.ref, i, n, ref);
    if (p.mask != nullptr) load_tokens(p.mask, i, n, mask);
    if (p.per_token) load_tokens(p.adv, i, n, adv);
  }
  float a;  // of the sequence
  __device__ __forceinline__ void sequence(int s) {
    if (!p.per_token) a = p.adv[s];
  }
  __device__ __forceinline__ void add(int j, Sums& sum) const {
    if (p.mask != nullptr && !mask[j]) return;
    const float at = p.per_token ? adv[j] : a;
    const double d = static_cast<double>(old_nll[j]) - static_cast<double>(nll[j]);
    const bool cut = p.clipped(at, d);
    float token = cut ? -(at > 0.0f ? p.r_high : p.r_low) * at : -PolicyArgs::ratio(at, d);
    if (p.ref != nullptr) {
      float em1, k;
      exp_terms(nll[j] - ref[j], em1, k);
      if (p.kl_weight != 0.0f) token = __builtin_fmaf(p.kl_weight, k, token);
      sum.b += k;
    }
    sum.a += token;
    sum.c += 1;
    sum.d += cut;
  }
};

struct PreferenceTerms {
  const float *nll_p, *ref_p;
  const uint8_t* mask_p;
  float nll[kPer], ref[kPer];
  uint8_t mask[kPer];
  __device__ __forceinline__ void load(int64_t i, int64_t n) {
    load_tokens(nll_p, i, n, nll);
    if (ref_p != nullptr) load_tokens(ref_p, i, n, ref);
    if (mask_p != nullptr) load_tokens(mask_p, i, n, mask);
  }
  __device__ __forceinline__ void sequence(int) {}
  __device__ __forceinline__ void add(int j, Sums& sum) const {
    if (mask_p != nullptr && !mask[j]) return;
    sum.a += (ref_p != nullptr ? static_cast<double>(ref[j]) : 0.0) - static_cast<double>(nll[j]);
    sum.c += 1;
  }
};

template <typename Terms>
__global__ __launch_bounds__(kThreads) void k_seq_sums(Terms w, Offsets off, int64_t span,
                                                       Sums* __restrict__ head,
                                                       Sums* __restrict__ carry) {
  __shared__ int marks[kWaves][kTile];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kWaves + wave;
  const int64_t n = off.n, t0 = at * span, t1 = min(t0 + span, n);
  if (t0 >= n) return;
  const Sums none{0.0, 0.0, 0, 0};
  Sums open = none;    // the lane's part of the sequence that the tile starts within
  bool fresh = false;  // whether that sequence started in this span
  Walk walk;
  walk.find(off, static_cast<int>(t0), lane);
  auto valid = [&](int s) { return s >= 0 && s < off.count; };
  for (int64_t tile0 = t0; tile0 < t1; tile0 += kTile) {
    w.load(tile0 + lane * kPer, n);
    int start[kPer], s;
    const bool any = walk.tile(off, static_cast<int>(tile0), lane, marks[wave], start, s);
    // tokens past n are in no sequence: off.n ends the last one at the latest
    const int left = static_cast<int>(min(n - tile0, static_cast<int64_t>(kTile))) - lane * kPer;
    if (!any) {
      if (valid(s)) {
        w.sequence(s);
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (j < left) w.add(j, open);
      }
      continue;
    }
    // the lane's tokens before its first start, those behind its last, and
    // the sequences between them, whole
    Sums lead = none, sum = none;
    bool has = false;
    int first = s;
    if (valid(s)) w.sequence(s);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (start[j] >= 0) {
        if (!has) lead = sum;
        else if (valid(s)) head[s] = sum;
        has = true;
        sum = none;
        s = start[j];
        if (valid(s)) w.sequence(s);
      }
      if (j < left && valid(s)) w.add(j, sum);
    }
    open.template join<64>();
    // inclusive scan of the parts since the last start
    Sums scan = sum;
    bool seen = has;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const Sums u = scan.up(o);
      const bool us = __shfl_up(static_cast<int>(seen), o, 64);
      if (lane >= o && !seen) {
        scan.add(u);
        seen = us;
      }
    }
    // what the lane's first start ends
    Sums end = scan.up(1);
    bool inside = __shfl_up(static_cast<int>(seen), 1, 64);
    if (lane == 0) {
      end = none;
      inside = false;
    }
    if (!inside) {
      Sums o = open;
      o.add(end);
      end = o;
    }
    end.add(lead);
    if (has) {
      if (inside || fresh) {
        if (valid(first)) head[first] = end;
      } else {
        carry[at] = end;
      }
    }
    // (a start in the tile: the last lane has seen one)
    open = lane == 63 ? scan : none;
    fresh = true;
  }
  open.template join<64>();
  if (lane != 0) return;
  if (!fresh) carry[at] = open;
  else if (valid(walk.next - 1)) head[walk.next - 1] = open;
}

// A sequence's sums: its part in the span where it starts and the carries of
// the spans behind, G lanes.
template <int G>
__device__ __forceinline__ Sums sequence_sums(const Offsets& off, int s, int64_t span,
                                              const Sums* __restrict__ head,
                                              const Sums* __restrict__ carry) {
  Sums sum{0.0, 0.0, 0, 0};
  const int l = threadIdx.x % G;
  if (s < off.count) {
    const int lo = off.at(s), hi = off.at(s + 1);
    if (lo < hi) {
      if (l == 0) sum = head[s];
      const int64_t last = (hi - 1) / span;
      for (int64_t k = lo / span + 1 + l; k <= last; k += G) sum.add(carry[k]);
    }
  }
  sum.template join<G>();
  return sum;
}

struct PolicyOut {
  float *loss, *kl;
  int32_t *count, *clipped;
  int mean;
};
template <int G>
__global__ __launch_bounds__(kThreads) void k_policy_join(Offsets off, int64_t span,
                                                          const Sums* __restrict__ head,
                                                          const Sums* __restrict__ carry,
                                                          PolicyOut o) {
  const int s = blockIdx.x * (kThreads / G) + threadIdx.x / G;
  const Sums sum = sequence_sums<G>(off, s, span, head, carry);
  if (s >= off.count || threadIdx.x % G != 0) return;
  const double part = o.mean ? 1.0 / max(sum.c, 1) : 1.0;
  o.loss[s] = static_cast<float>(sum.a * part);
  o.kl[s] = static_cast<float>(sum.b * part);
  o.count[s] = sum.c;
  o.clipped[s] = sum.d;
}

struct PreferenceHow {
  int kind, mean;
  float beta, margin, smoothing;
};
// f(x)
__device__ __forceinline__ double preference(const PreferenceHow& h, double x) {
  if (h.kind == MUON_PREFERENCE_HINGE) return x < 1.0 ? 1.0 - x : (x >= 1.0 ? 0.0 : x);
  if (h.kind == MUON_PREFERENCE_SQUARED) return (1.0 - x) * (1.0 - x);
  // (1 - smoothing) softplus(-x) + smoothing softplus(x); no 0 inf
  const double soft = log1p(exp(-fabs(x)));
  double f = 0.0;
  if (h.smoothing != 1.0f) f += (1.0 - h.smoothing) * (soft + (x < 0.0 ? -x : 0.0));
  if (h.smoothing != 0.0f) f += h.smoothing * (soft + (x > 0.0 ? x : 0.0));
  return f;
}
// f'(x)
__device__ __forceinline__ float preference_slope(const PreferenceHow& h, float x) {
  if (h.kind == MUON_PREFERENCE_HINGE) return x < 1.0f ? -1.0f : (x >= 1.0f ? 0.0f : x);
  if (h.kind == MUON_PREFERENCE_SQUARED) return 2.0f * (x - 1.0f);
  return h.smoothing - 1.0f / (1.0f + expf(x));
}

struct PreferenceOut {
  float *loss, *margin, *reward;
  int32_t* count;
};
template <int G>
__global__ __launch_bounds__(kThreads) void k_preference_join(Offsets off, int64_t span,
                                                              const Sums* __restrict__ head,
                                                              const Sums* __restrict__ carry,
                                                              PreferenceHow h, PreferenceOut o) {
  const int i = blockIdx.x * (kThreads / G) + threadIdx.x / G;
  const int pairs = off.count / 2;
  double reward[2];
  int count[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const Sums sum = sequence_sums<G>(off, i < pairs ? 2 * i + k : off.count, span, head, carry);
    reward[k] = h.beta * sum.a;
    if (h.mean) reward[k] /= max(sum.c, 1);
    count[k] = sum.c;
  }
  if (i >= pairs || threadIdx.x % G != 0) return;
  const double x = reward[0] - reward[1] - h.margin;
  o.margin[i] = static_cast<float>(x);
  o.loss[i] = count[0] > 0 && count[1] > 0 ? static_cast<float>(preference(h, x)) : 0.0f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    o.reward[2 * i + k] = static_cast<float>(reward[k]);
    o.count[2 * i + k] = count[k];
  }
}

struct PolicySlope {
  PolicyTerms w;
  const float* dloss;
  const int32_t* count;
  int mean;
  float each;
  __device__ __forceinline__ void load(int64_t i, int64_t n) { w.load(i, n); }
  __device__ __forceinline__ void sequence(int s) {
    w.sequence(s);
    each = dloss[s];
    if (mean) each /= static_cast<float>(max(count[s], 1));
  }
  __device__ __forceinline__ float slope(int j) const {
    if (w.p.mask != nullptr && !w.mask[j]) return 0.0f;
    const float at = w.p.per_token ? w.adv[j] : w.a;
    const double d = static_cast<double>(w.old_nll[j]) - static_cast<double>(w.nll[j]);
    float g = w.p.clipped(at, d) ? 0.0f : PolicyArgs::ratio(at, d);
    if (w.p.kl_weight != 0.0f) {
      float em1, k;
      exp_terms(w.nll[j] - w.ref[j], em1, k);
      g = __builtin_fmaf(w.p.kl_weight, em1, g);
    }
    return each * g;
  }
};

struct PreferenceSlope {
  const float *margin, *dloss;
  const int32_t* count;
  const uint8_t* mask_p;
  PreferenceHow h;
  float each;
  uint8_t mask[kPer];
  __device__ __forceinline__ void load(int64_t i, int64_t n) {
    if (mask_p != nullptr) load_tokens(mask_p, i, n, mask);
  }
  __device__ __forceinline__ void sequence(int s) {
    const int i = s >> 1, mine = count[s];
    if (mine <= 0 || count[s ^ 1] <= 0) {
      each = 0.0f;
      return;
    }
    const float g = h.beta * dloss[i] * preference_slope(h, margin[i]);
    each = (s & 1) != 0 ? g : -g;
    if (h.mean) each /= static_cast<float>(mine);
  }
  __device__ __forceinline__ float slope(int j) const {
    return mask_p != nullptr && !mask[j] ? 0.0f : each;
  }
};

// dnll of the tokens that are in a sequence.
template <typename Slope>
__global__ __launch_bounds__(kThreads) void k_seq_slopes(Slope w, Offsets off, int64_t span,
                                                         float* __restrict__ dnll) {
  __shared__ int marks[kWaves][kTile];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWaves + wave) * span;
  const int64_t n = off.n, t1 = min(t0 + span, n);
  if (t0 >= n) return;
  Walk walk;
  walk.find(off, static_cast<int>(t0), lane);
  auto valid = [&](int s) { return s >= 0 && s < off.count; };
  for (int64_t tile0 = t0; tile0 < t1; tile0 += kTile) {
    const int64_t i = tile0 + lane * kPer;
    w.load(i, n);
    int start[kPer], s;
    walk.tile(off, static_cast<int>(tile0), lane, marks[wave], start, s);
    float g[kPer];
    bool write[kPer], all = i + kPer <= n;
    if (valid(s)) w.sequence(s);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (start[j] >= 0) {
        s = start[j];
        if (valid(s)) w.sequence(s);
      }
      write[j] = i + j < n && valid(s);
      all &= write[j];
      g[j] = write[j] ? w.slope(j) : 0.0f;
    }
    if (all) {
      __builtin_memcpy(dnll + i, g, sizeof(g));
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (write[j]) dnll[i + j] = g[j];
    }
  }
}

// -------------------------------------------------------------------- host

// Waves of a launch: eight to a SIMD.
constexpr int64_t kSpans = 8192;
constexpr int64_t kMaxSequences = static_cast<int64_t>(1) << 24;

int64_t span_of(int64_t n) { return (n + kSpans * kTile - 1) / (kSpans * kTile) * kTile; }
int64_t spans_of(int64_t n) { return n == 0 ? 0 : (n + span_of(n) - 1) / span_of(n); }

struct SeqWs {
  size_t head, carry, total;
};
SeqWs seq_ws(int64_t n, int64_t sequences) {
  SeqWs w{};
  w.head = 0;
  w.carry = align256(static_cast<size_t>(sequences) * sizeof(Sums));
  w.total = w.carry + align256(static_cast<size_t>(spans_of(n)) * sizeof(Sums));
  return w;
}

int check_sequences(int64_t n, int64_t sequences) {
  if (n < 0 || n > kMaxTokens) return set_error(MUON_ERR_BAD_SHAPE, "n must be in [0, 2^26)");
  if (sequences < 0 || sequences > kMaxSequences)
    return set_error(MUON_ERR_BAD_SHAPE, "sequences must be in [0, 2^24]");
  return MUON_OK;
}
int check_seq_ws(const void* ws, size_t bytes, size_t need, const char* who) {
  if (ws == nullptr || bytes < need || reinterpret_cast<uintptr_t>(ws) % 256 != 0)
    return set_error(MUON_ERR_WORKSPACE_TOO_SMALL, std::string(who) + " needs " +
                                                       std::to_string(need) +
                                                       " bytes of workspace, 256-byte aligned");
  return MUON_OK;
}
int check_policy(const PolicyArgs& p, const void* offsets, double clip_low, double clip_high,
                 int64_t n) {
  if (!(clip_low >= 0.0 && clip_low <= 1.0) || !(clip_high >= 0.0 && std::isfinite(clip_high)))
    return set_error(MUON_ERR_INVALID_ARG, "clip_low must be in [0, 1], clip_high finite and >= 0");
  if (!std::isfinite(p.kl_weight))
    return set_error(MUON_ERR_INVALID_ARG, "kl_weight must be finite");
  if (offsets == nullptr || (p.adv == nullptr && (n > 0 || !p.per_token)) ||
      (n > 0 && (p.nll == nullptr || p.old_nll == nullptr)))
    return set_error(MUON_ERR_INVALID_ARG, "nll, old_nll, advantages or offsets is null");
  if (p.kl_weight != 0.0f && n > 0 && p.ref == nullptr)
    return set_error(MUON_ERR_INVALID_ARG, "kl_weight needs ref_nll");
  return MUON_OK;
}
PolicyArgs policy_args(const float* nll, const float* old_nll, const float* ref_nll,
                       const uint8_t* mask, const float* advantages, int32_t per_token,
                       double clip_low, double clip_high, float kl_weight) {
  PolicyArgs p{};
  p.nll = nll;
  p.old_nll = old_nll;
  p.ref = ref_nll;
  p.adv = advantages;
  p.mask = mask;
  p.d_low = std::log1p(-clip_low);  // -inf for 1
  p.d_high = std::log1p(clip_high);
  p.r_low = static_cast<float>(1.0 - clip_low);
  p.r_high = static_cast<float>(1.0 + clip_high);
  p.kl_weight = kl_weight;
  p.per_token = per_token != 0;
  return p;
}
int check_preference(int64_t sequences, int32_t kind, float beta, float margin, float smoothing) {
  if (sequences % 2 != 0)
    return set_error(MUON_ERR_BAD_SHAPE, "sequences must be even: two to a pair");
  if (kind != MUON_PREFERENCE_LOGISTIC && kind != MUON_PREFERENCE_HINGE &&
      kind != MUON_PREFERENCE_SQUARED)
    return set_error(MUON_ERR_INVALID_ARG, "unknown kind of preference loss");
  if (!std::isfinite(beta) || !std::isfinite(margin))
    return set_error(MUON_ERR_INVALID_ARG, "beta and margin must be finite");
  if (!(smoothing >= 0.0f && smoothing <= 1.0f) ||
      (smoothing != 0.0f && kind != MUON_PREFERENCE_LOGISTIC))
    return set_error(MUON_ERR_INVALID_ARG, "smoothing must be in [0, 1], and 0 but for logistic");
  return MUON_OK;
}

template <typename Terms>
void launch_sums(const Terms& w, const Offsets& off, Sums* head, Sums* carry, hipStream_t s) {
  const int64_t blocks = (spans_of(off.n) + kWaves - 1) / kWaves;
  if (blocks > 0)
    hipLaunchKernelGGL(k_seq_sums<Terms>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s,
                       w, off, span_of(off.n), head, carry);
}
template <typename Slope>
void launch_slopes(const Slope& w, const Offsets& off, float* dnll, hipStream_t s) {
  const int64_t blocks = (spans_of(off.n) + kWaves - 1) / kWaves;
  hipLaunchKernelGGL(k_seq_slopes<Slope>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s,
                     w, off, span_of(off.n), dnll);
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

size_t sequence_loss_workspace_size(int64_t n, int64_t sequences) {
  if (check_sequences(n, sequences) != MUON_OK || sequences == 0) return 0;
  return seq_ws(n, sequences).total;
}

int policy_loss_forward(const float* nll, const float* old_nll, const float* ref_nll,
                        const uint8_t* mask, const float* advantages, int32_t per_token,
                        const int32_t* offsets, int64_t sequences, int64_t n, double clip_low,
                        double clip_high, float kl_weight, int32_t mean, float* loss, float* kl,
                        int32_t* count, int32_t* clipped, void* workspace, size_t workspace_bytes,
                        hipStream_t stream) {
  int rc = check_sequences(n, sequences);
  if (rc != MUON_OK) return rc;
  if (sequences == 0) return MUON_OK;
  const PolicyArgs p = policy_args(nll, old_nll, ref_nll, mask, advantages, per_token, clip_low,
                                   clip_high, kl_weight);
  if ((rc = check_policy(p, offsets, clip_low, clip_high, n)) != MUON_OK) return rc;
  if (loss == nullptr || kl == nullptr || count == nullptr || clipped == nullptr)
    return set_error(MUON_ERR_INVALID_ARG, "loss, kl, count or clipped is null");
  const SeqWs w = seq_ws(n, sequences);
  if ((rc = check_seq_ws(workspace, workspace_bytes, w.total, "policy_loss_forward")) != MUON_OK)
    return rc;
  Sums* head = reinterpret_cast<Sums*>(static_cast<char*>(workspace) + w.head);
  Sums* carry = reinterpret_cast<Sums*>(static_cast<char*>(workspace) + w.carry);
  const Offsets off{offsets, static_cast<int>(sequences), static_cast<int>(n)};
  PolicyTerms terms{};
  terms.p = p;
  launch_sums(terms, off, head, carry, stream);
  const unsigned blocks = static_cast<unsigned>((sequences + kWaves - 1) / kWaves);
  hipLaunchKernelGGL(k_policy_join<64>, dim3(blocks), dim3(kThreads), 0, stream, off,
                     std::max<int64_t>(span_of(n), 1), head, carry,
                     PolicyOut{loss, kl, count, clipped, mean != 0});
  return check_launch("policy loss launch");
}

int policy_loss_backward(const float* nll, const float* old_nll, const float* ref_nll,
                         const uint8_t* mask, const float* advantages, int32_t per_token,
                         const int32_t* offsets, int64_t sequences, int64_t n, double clip_low,
                         double clip_high, float kl_weight, int32_t mean, const int32_t* count,
                         const float* dloss, float* dnll, hipStream_t stream) {
  int rc = check_sequences(n, sequences);
  if (rc != MUON_OK) return rc;
  if (sequences == 0 || n == 0) return MUON_OK;
  const PolicyArgs p = policy_args(nll, old_nll, ref_nll, mask, advantages, per_token, clip_low,
                                   clip_high, kl_weight);
  if ((rc = check_policy(p, offsets, clip_low, clip_high, n)) != MUON_OK) return rc;
  if (count == nullptr || dloss == nullptr || dnll == nullptr)
    return set_error(MUON_ERR_INVALID_ARG, "count, dloss or dnll is null");
  PolicySlope slope{};
  slope.w.p = p;
  if (kl_weight == 0.0f) slope.w.p.ref = nullptr;
  slope.dloss = dloss;
  slope.count = count;
  slope.mean = mean != 0;
  launch_slopes(slope, Offsets{offsets, static_cast<int>(sequences), static_cast<int>(n)}, dnll,
                stream);
  return check_launch("policy loss gradient launch");
}

int preference_loss_forward(const float* nll, const float* ref_nll, const uint8_t* mask,
                            const int32_t* offsets, int64_t sequences, int64_t n, int32_t kind,
                            float beta, float margin, float smoothing, int32_t mean, float* loss,
                            float* margins, float* reward, int32_t* count, void* workspace,
                            size_t workspace_bytes, hipStream_t stream) {
  int rc = check_sequences(n, sequences);
  if (rc != MUON_OK) return rc;
  if ((rc = check_preference(sequences, kind, beta, margin, smoothing)) != MUON_OK) return rc;
  if (sequences == 0) return MUON_OK;
  if (offsets == nullptr || (n > 0 && nll == nullptr))
    return set_error(MUON_ERR_INVALID_ARG, "nll or offsets is null");
  if (loss == nullptr || margins == nullptr || reward == nullptr || count == nullptr)
    return set_error(MUON_ERR_INVALID_ARG, "loss, margins, reward or count is null");
  const SeqWs w = seq_ws(n, sequences);
  if ((rc = check_seq_ws(workspace, workspace_bytes, w.total, "preference_loss_forward")) != MUON_OK)
    return rc;
  Sums* head = reinterpret_cast<Sums*>(static_cast<char*>(workspace) + w.head);
  Sums* carry = reinterpret_cast<Sums*>(static_cast<char*>(workspace) + w.carry);
  const Offsets off{offsets, static_cast<int>(sequences), static_cast<int>(n)};
  PreferenceTerms terms{};
  terms.nll_p = nll;
  terms.ref_p = ref_nll;
  terms.mask_p = mask;
  launch_sums(terms, off, head, carry, stream);
  const unsigned blocks = static_cast<unsigned>((sequences / 2 + kWaves - 1) / kWaves);
  hipLaunchKernelGGL(k_preference_join<64>, dim3(blocks), dim3(kThreads), 0, stream, off,
                     std::max<int64_t>(span_of(n), 1), head, carry,
                     PreferenceHow{kind, mean != 0, beta, margin, smoothing},
                     PreferenceOut{loss, margins, reward, count});
  return check_launch("preference loss launch");
}

int preference_loss_backward(const uint8_t* mask, const int32_t* offsets, int64_t sequences,
                             int64_t n, int32_t kind, float beta, float smoothing, int32_t mean,
                             const float* margins, const int32_t* count, const float* dloss,
                             float* dnll, hipStream_t stream) {
  int rc = check_sequences(n, sequences);
  if (rc != MUON_OK) return rc;
  if ((rc = check_preference(sequences, kind, beta, 0.0f, smoothing)) != MUON_OK) return rc;
  if (sequences == 0 || n == 0) return MUON_OK;
  if (offsets == nullptr || margins == nullptr || count == nullptr || dloss == nullptr ||
      dnll == nullptr)
    return set_error(MUON_ERR_INVALID_ARG, "offsets, margins, count, dloss or dnll is null");
  PreferenceSlope slope{};
  slope.margin = margins;
  slope.dloss = dloss;
  slope.count = count;
  slope.mask_p = mask;
  slope.h = PreferenceHow{kind, mean != 0, beta, 0.0f, smoothing};
  launch_slopes(slope, Offsets{offsets, static_cast<int>(sequences), static_cast<int>(n)}, dnll,
                stream);
  return check_launch("preference loss gradient launch");
}

}  // extern "C"
