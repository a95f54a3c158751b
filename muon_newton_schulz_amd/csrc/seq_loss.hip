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
#include <type_traits>

#include "train_common.h"

namespace muon {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kPer = 8, kTile = 64 * kPer;  // tokens of a lane, of a wave's tile

// count + 1 offsets, non-decreasing; whatever they hold, values are within
// [0, n].
struct Offsets {
  const int32_t* p;
  int count, n;  // sequences, tokens
  __device__ __forceinline__ int at(int s) const { return min(max(p[s], 0), n); }
};

// A lane's value from a lane before it (dpp: in registers, without the LDS
// trip of a shuffle); `none` where there is none.
enum : int { kShr1 = 0x111, kShr2 = 0x112, kShr4 = 0x114, kShr8 = 0x118, kWaveShr1 = 0x138,
             kBcast15 = 0x142, kBcast31 = 0x143 };
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp(int x, int none) {
  return __builtin_amdgcn_update_dpp(none, x, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double x) {
  const int2 v = __builtin_bit_cast(int2, x);
  return __builtin_bit_cast(double, int2{dpp<CTRL, ROWS>(v.x, 0), dpp<CTRL, ROWS>(v.y, 0)});
}
// f over the steps of an inclusive scan of the wave: 1, 2, 4 and 8 lanes within
// rows of 16, then rows 0 and 2 into the next, then the first half into the
// second.
template <typename F>
__device__ __forceinline__ void scan_steps(F&& f) {
  f(std::integral_constant<int, kShr1>{}, std::integral_constant<int, 0xf>{});
  f(std::integral_constant<int, kShr2>{}, std::integral_constant<int, 0xf>{});
  f(std::integral_constant<int, kShr4>{}, std::integral_constant<int, 0xf>{});
  f(std::integral_constant<int, kShr8>{}, std::integral_constant<int, 0xf>{});
  f(std::integral_constant<int, kBcast15>{}, std::integral_constant<int, 0xa>{});
  f(std::integral_constant<int, kBcast31>{}, std::integral_constant<int, 0xc>{});
}
__device__ __forceinline__ double last_lane(double x) {
  const int2 v = __builtin_bit_cast(int2, x);
  return __builtin_bit_cast(double, int2{__builtin_amdgcn_readlane(v.x, 63),
                                         __builtin_amdgcn_readlane(v.y, 63)});
}

// The sequences of a lane's eight tokens, tile by tile.  A wave keeps 64
// offsets, one a lane, and what Source::of gives for their sequences, and loads
// others only when its tiles have passed them: a load a tile would be most of
// the time of a short span.
template <typename Source>
struct Walk {
  using Value = typename Source::Value;
  int next;      // the first sequence (count: the end) that starts at the tile or later
  int batch;     // lane's offset and value are those of sequence batch + lane
  int offset;
  Value value, prior;  // prior: of sequence batch - 1
  bool moved;          // whether the last tile went past the batch

  __device__ __forceinline__ static bool valid(const Offsets& off, int s) {
    return s >= 0 && s < off.count;
  }
  __device__ __forceinline__ void load(const Offsets& off, const Source& w, int first, int lane) {
    batch = first;
    offset = first + lane <= off.count ? off.at(first + lane) : off.n + kTile;
    value = valid(off, first + lane) ? w.of(first + lane) : Value{};
  }
  // 64-way search for the first offset from lo on that is not below `token`:
  // it is one of at most 64 from lo on, len of them
  __device__ __forceinline__ static void search(const Offsets& off, int token, int lane, int& lo,
                                                int& len) {
    len = off.count + 1 - lo;
    while (len > 64) {
      const int step = (len + 63) >> 6, q = lane * step + step - 1;
      const bool below = q < len && off.at(lo + q) < token;
      const int c = __popcll(__ballot(below));
      lo += c * step;
      len = min(step - 1, len - c * step);
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
  }
  __device__ __forceinline__ void find(const Offsets& off, const Source& w, int token, int lane) {
    int lo = 0, len;
    search(off, token, lane, lo, len);
    load(off, w, lo, lane);
    prior = valid(off, lo - 1) ? w.of(lo - 1) : Value{};
    next = lo + __popcll(__ballot(lane < len && offset < token));
  }
  // Past the sequences that start at `token` as the one before next does, and
  // are empty but for the last.
  __device__ __forceinline__ void skip(const Offsets& off, const Source& w, int token, int lane) {
    int lo = next, len;
    search(off, token + 1, lane, lo, len);
    next = lo + __popcll(__ballot(lane < len && off.at(lo + lane) <= token));
    load(off, w, next, lane);
    prior = valid(off, next - 1) ? w.of(next - 1) : Value{};
  }
  // Marks the starts in the tile: start[j] is the sequence that starts at the
  // lane's token j, or -1; s: the one its first token is in unless it
  // starts there (-1 and count: none).  Returns whether any starts.
  __device__ __forceinline__ bool tile(const Offsets& off, const Source& w, int tile0, int lane,
                                       int* lds, int (&start)[kPer], int& s) {
    s = next - 1;
    moved = false;
    bool any = false;
    while (next <= off.count) {
      if (next >= batch + 64) {
        const int before = __builtin_amdgcn_readlane(offset, 63);
        prior = value.lane(63);
        load(off, w, next, lane);
        moved = any;
        // A whole batch that starts where the one before it ended is part of a
        // run of empty sequences (unused slots of a batch of fixed capacity),
        // of which only the last one's mark counts.  (Forward and backward of
        // 50001 tokens in 100 sequences, the other slots behind them, walked 64
        // at a time, each load waiting for the one before, and this way: 2^13
        // slots 58 and 88 us, 24 and 9; 2^20 9.3 and 12.6 ms, 0.39 and 0.01.)
        if (any && __builtin_amdgcn_readlane(offset, 63) == before) {
          skip(off, w, before, lane);
          const int o = before - tile0;
          if (lane == 0 && o >= 0 && o < kTile) atomicMax(&lds[o], next - 1);
        }
      }
      const int o = offset - tile0;
      const uint64_t in = __ballot(batch + lane >= next && o < kTile);
      if (in == 0) break;
      if (!any) {
        any = true;
#pragma unroll
        for (int j = 0; j < kPer; ++j) lds[lane * kPer + j] = -1;
        wave_sync();
      }
      // of several that start at a token all but the last are empty
      if ((in >> lane & 1) != 0 && o >= 0) atomicMax(&lds[o], batch + lane);
      next += __popcll(in);
      if (next < batch + 64) break;
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
    scan_steps([&](auto ctrl, auto rows) {
      last = max(last, dpp<decltype(ctrl)::value, decltype(rows)::value>(last, -1));
    });
    s = max(s, dpp<kWaveShr1, 0xf>(last, -1));
    return true;
  }
  // The values of the sequences that the lane's tokens of the last tile are
  // in, and which of the tokens are in one.  any, s, start: tile's.
  __device__ __forceinline__ int values(const Offsets& off, const Source& w, bool any, int s,
                                        const int (&start)[kPer], Value (&v)[kPer]) const {
    if (!any) {
      const Value x = value.lane(max(s - batch, 0)), y = s < batch ? prior : x;
#pragma unroll
      for (int j = 0; j < kPer; ++j) v[j] = y;
      return valid(off, s) ? 0xff : 0;
    }
    int in = 0;
    if (!moved) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        s = max(s, start[j]);
        const Value x = value.lane(max(s - batch, 0));
        v[j] = s < batch ? prior : x;
        in |= static_cast<int>(valid(off, s)) << j;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        s = max(s, start[j]);
        v[j] = valid(off, s) ? w.of(s) : Value{};
        in |= static_cast<int>(valid(off, s)) << j;
      }
    }
    return in;
  }
};

// What a walk keeps of a sequence: nothing, or some fp32 values.
struct Nothing {
  __device__ __forceinline__ Nothing lane(int) const { return {}; }
};
struct One {
  float a;
  __device__ __forceinline__ One lane(int l) const { return {__shfl(a, l, 64)}; }
};
struct Two {
  float a, b;
  __device__ __forceinline__ Two lane(int l) const { return {__shfl(a, l, 64), __shfl(b, l, 64)}; }
};

// A lane's tokens.
struct Tokens {
  float nll[kPer], old_nll[kPer], ref[kPer], adv[kPer];
  uint8_t mask[kPer];
};
// Eight values from token i on; WHOLE: all of them below n, else the last one
// in place of those past it.
template <bool WHOLE, typename T>
__device__ __forceinline__ void load_values(const T* p, int i, int n, T (&v)[kPer]) {
  if constexpr (WHOLE) {
    __builtin_memcpy(v, p + static_cast<uint32_t>(i), sizeof(v));
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] = p[static_cast<uint32_t>(min(i + j, n - 1))];
  }
}
template <typename Source>
__device__ __forceinline__ void load_tile(const Source& w, int tile0, int lane, int n, Tokens& t) {
  if (tile0 + kTile <= n) w.template load<true>(tile0 + lane * kPer, n, t);
  else w.template load<false>(tile0 + lane * kPer, n, t);
}
// Which of eight tokens from i on are below n and not masked.
__device__ __forceinline__ int counting(const Tokens& t, const uint8_t* mask, int i, int n) {
  int in = i + kPer <= n ? 0xff : (1 << max(n - i, 0)) - 1;
  if (mask != nullptr) {
    int m = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) m |= (t.mask[j] != 0 ? 1 : 0) << j;
    in &= m;
  }
  return in;
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
  // those of a lane before, 0 where there is none
  template <int CTRL, int ROWS>
  __device__ __forceinline__ Sums before() const {
    return {dpp<CTRL, ROWS>(a), dpp<CTRL, ROWS>(b), dpp<CTRL, ROWS>(c, 0), dpp<CTRL, ROWS>(d, 0)};
  }
  __device__ __forceinline__ Sums last() const {
    return {last_lane(a), last_lane(b), __builtin_amdgcn_readlane(c, 63),
            __builtin_amdgcn_readlane(d, 63)};
  }
  template <int G>
  __device__ __forceinline__ void join() {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1)
      add({__shfl_xor(a, o, 64), __shfl_xor(b, o, 64), __shfl_xor(c, o, 64), __shfl_xor(d, o, 64)});
  }
};

// e^x - 1 and e^x - 1 - x of eight values.  The second is a difference of near
// values, which a polynomial replaces below |x| = 1/2: x^2 (1/2 + x / 6 + ... +
// x^6 / 40320), off by 2 x^7 / 9! < 2^-24 of itself.
__device__ __forceinline__ void exp_terms(const float (&x)[kPer], float (&em1)[kPer],
                                          float (&k)[kPer]) {
  bool far = false;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    float p = 1.0f / 40320.0f;
    p = __builtin_fmaf(p, x[j], 1.0f / 5040.0f);
    p = __builtin_fmaf(p, x[j], 1.0f / 720.0f);
    p = __builtin_fmaf(p, x[j], 1.0f / 120.0f);
    p = __builtin_fmaf(p, x[j], 1.0f / 24.0f);
    p = __builtin_fmaf(p, x[j], 1.0f / 6.0f);
    p = __builtin_fmaf(p, x[j], 0.5f);
    k[j] = x[j] * x[j] * p;
    em1[j] = x[j] + k[j];
    far |= !(fabsf(x[j]) < 0.5f);
  }
  if (__ballot(far) == 0) return;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const float e = expf(x[j]) - 1.0f;
    if (!(fabsf(x[j]) < 0.5f)) {
      em1[j] = e;
      k[j] = e - x[j];
    }
  }
}

struct PolicyArgs {
  const float *nll, *old_nll, *ref, *adv;
  const uint8_t* mask;
  // The clip as bounds of d: r > 1 + hi where d > log(1 + hi).  (The exact
  // difference against the fp64 bound: a ratio next to the border is on its own
  // side of it.)
  double d_low, d_high;
  float f_low, f_high;  // the bounds rounded to fp32
  float r_low, r_high, kl_weight;
  int per_token;

  template <bool WHOLE>
  __device__ __forceinline__ void load(int i, int n, Tokens& t) const {
    load_values<WHOLE>(nll, i, n, t.nll);
    load_values<WHOLE>(old_nll, i, n, t.old_nll);
    if (ref != nullptr) load_values<WHOLE>(ref, i, n, t.ref);
    if (mask != nullptr) load_values<WHOLE>(mask, i, n, t.mask);
    if (per_token) load_values<WHOLE>(adv, i, n, t.adv);
  }
  // Which of the tokens the clip holds, and the ratios (0 where A is, so
  // that no 0 inf comes of a ratio beyond fp32; a NaN stays one).  Rounding
  // keeps the order, so unless d rounds to what the bound rounds to, fp32
  // decides as the exact difference does.
  __device__ __forceinline__ int ratios(const Tokens& t, const float (&a)[kPer],
                                        float (&r)[kPer]) const {
    int cut = 0;
    bool border = false;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const float d = t.old_nll[j] - t.nll[j];
      const bool up = a[j] > 0.0f;
      cut |= static_cast<int>(up ? d > f_high : a[j] < 0.0f && d < f_low) << j;
      border |= d == (up ? f_high : f_low);
      r[j] = a[j] == 0.0f && d == d ? 0.0f : expf(d);
    }
    if (__ballot(border) == 0) return cut;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const double e = static_cast<double>(t.old_nll[j]) - static_cast<double>(t.nll[j]);
      const bool c = a[j] > 0.0f ? e > d_high : a[j] < 0.0f && e < d_low;
      cut = (cut & ~(1 << j)) | static_cast<int>(c) << j;
    }
    return cut;
  }
  __device__ __forceinline__ void kl(const Tokens& t, float (&em1)[kPer], float (&k)[kPer]) const {
    float x[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) x[j] = t.nll[j] - t.ref[j];
    exp_terms(x, em1, k);
  }
};

struct PolicyTerms {
  PolicyArgs p;
  using Value = One;  // the sequence's advantage
  __device__ __forceinline__ Value of(int s) const { return {p.per_token ? 0.0f : p.adv[s]}; }
  __device__ __forceinline__ const uint8_t* mask() const { return p.mask; }
  template <bool WHOLE>
  __device__ __forceinline__ void load(int i, int n, Tokens& t) const {
    p.load<WHOLE>(i, n, t);
  }
  // What a token adds to its sequence's sums.
  struct Term {
    float a, b;
    int n;  // tokens, and << 16 those that the clip holds
  };
  // Sum of at most a lane's eight, in fp64 as all sums: neighbours cancel too
  // (policy step of 33.5 M tokens 216 us, with fp32 here 215).
  struct Part {
    double a, b;
    int n;
    __device__ __forceinline__ Sums sums() const { return {a, b, n & 0xffff, n >> 16}; }
    __device__ __forceinline__ Part operator+(const Term& o) const {
      return {a + o.a, b + o.b, n + o.n};
    }
  };
  __device__ __forceinline__ void terms(const Tokens& t, int in, const Value (&v)[kPer],
                                        Term (&r)[kPer]) const {
    float a[kPer], ratio[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) a[j] = p.per_token ? t.adv[j] : v[j].a;
    const int cut = p.ratios(t, a, ratio);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool c = (cut >> j) & 1;
      r[j].a = -(c ? (a[j] > 0.0f ? p.r_high : p.r_low) : ratio[j]) * a[j];
      r[j].b = 0.0f;
      r[j].n = c ? 0x10001 : 1;
    }
    if (p.ref != nullptr) {
      float em1[kPer], k[kPer];
      p.kl(t, em1, k);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        r[j].b = k[j];
        if (p.kl_weight != 0.0f) r[j].a = __builtin_fmaf(p.kl_weight, k[j], r[j].a);
      }
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (((in >> j) & 1) == 0) r[j] = Term{0.0f, 0.0f, 0};
  }
};

struct PreferenceTerms {
  const float *nll, *ref;
  const uint8_t* mask_p;
  using Value = Nothing;
  __device__ __forceinline__ Value of(int) const { return {}; }
  __device__ __forceinline__ const uint8_t* mask() const { return mask_p; }
  template <bool WHOLE>
  __device__ __forceinline__ void load(int i, int n, Tokens& t) const {
    load_values<WHOLE>(nll, i, n, t.nll);
    if (ref != nullptr) load_values<WHOLE>(ref, i, n, t.ref);
    if (mask_p != nullptr) load_values<WHOLE>(mask_p, i, n, t.mask);
  }
  // fp64 throughout: the sum is multiplied by beta and stands in an exponent
  struct Term {
    double a;
    int n;
    __device__ __forceinline__ Sums sums() const { return {a, 0.0, n, 0}; }
    __device__ __forceinline__ Term operator+(const Term& o) const { return {a + o.a, n + o.n}; }
  };
  using Part = Term;
  __device__ __forceinline__ void terms(const Tokens& t, int in, const Value (&)[kPer],
                                        Term (&r)[kPer]) const {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const double a = (ref != nullptr ? static_cast<double>(t.ref[j]) : 0.0) -
                       static_cast<double>(t.nll[j]);
      r[j] = ((in >> j) & 1) != 0 ? Term{a, 1} : Term{0.0, 0};
    }
  }
};

// The sums of span `at`, by a wave.
template <typename Terms>
__device__ __forceinline__ void span_sums(const Terms& w, const Offsets& off, int span, int at,
                                          int lane, int* marks, Sums* head, Sums* carry) {
  using Term = typename Terms::Term;
  using Part = typename Terms::Part;
  const int n = off.n, t0 = at * span, t1 = min(t0 + span, n);
  if (t0 >= n) return;
  const Sums none{0.0, 0.0, 0, 0};
  // the part of the sequence that the tile starts within: spread over the
  // lanes, or the last lane's alone
  Sums open = none;
  bool spread = false;
  bool fresh = false;  // whether that sequence started in this span
  auto valid = [&](int s) { return s >= 0 && s < off.count; };
  auto whole = [&]() {  // open as a whole, in every lane
    if (spread)
      scan_steps([&](auto ctrl, auto rows) {
        open.add(open.template before<decltype(ctrl)::value, decltype(rows)::value>());
      });
    open = open.last();
  };
  Tokens tok;
  load_tile(w, t0, lane, n, tok);
  Walk<Terms> walk;
  walk.find(off, w, t0, lane);
  for (int tile0 = t0; tile0 < t1; tile0 += kTile) {
    int start[kPer], s;
    const bool any = walk.tile(off, w, tile0, lane, marks, start, s);
    typename Terms::Value v[kPer];
    Term r[kPer];
    const int in = walk.values(off, w, any, s, start, v) &
                   counting(tok, w.mask(), tile0 + lane * kPer, n);
    w.terms(tok, in, v, r);
    // (the next tile's loads run during the sums below)
    if (tile0 + kTile < t1) load_tile(w, tile0 + kTile, lane, n, tok);
    if (!any) {
      Part sum{};
#pragma unroll
      for (int j = 0; j < kPer; ++j) sum = sum + r[j];
      open.add(sum.sums());
      spread = true;
      continue;
    }
    // the lane's tokens before its first start, and those from its last on
    Part lead{}, sum{};
    int starts = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool here = start[j] >= 0;
      if (here && starts == 0) lead = sum;
      if (here) sum = Part{};
      starts += here;
      sum = sum + r[j];
    }
    // the sequences between them, whole
    if (__ballot(starts > 1) != 0) {
      Part part{};
      int q = -1;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (start[j] >= 0) {
          if (valid(q)) head[q] = part.sums();
          q = start[j];
          part = Part{};
        }
        part = part + r[j];
      }
    }
    whole();
    // inclusive scan of the parts since the last start
    Sums scan = sum.sums();
    int seen = starts > 0;
    scan_steps([&](auto ctrl, auto rows) {
      constexpr int C = decltype(ctrl)::value, R = decltype(rows)::value;
      const Sums u = scan.template before<C, R>();
      const int us = dpp<C, R>(seen, 0);
      if (!seen) scan.add(u);
      seen |= us;
    });
    // what the lane's first start ends
    Sums end = scan.template before<kWaveShr1, 0xf>();
    const bool inside = dpp<kWaveShr1, 0xf>(seen, 0) != 0;
    if (!inside) end.add(open);
    end.add(lead.sums());
    if (starts > 0) {
      if (inside || fresh) {
        if (valid(s)) head[s] = end;
      } else {
        carry[at] = end;
      }
    }
    // (with a start in the tile, the last lane has seen one)
    open = lane == 63 ? scan : none;
    spread = false;
    fresh = true;
  }
  whole();
  if (lane != 0) return;
  if (!fresh) carry[at] = open;
  else if (valid(walk.next - 1)) head[walk.next - 1] = open;
}

template <typename Terms>
__global__ __launch_bounds__(kThreads) void k_seq_sums(Terms w, Offsets off, int span,
                                                       Sums* __restrict__ head,
                                                       Sums* __restrict__ carry) {
  __shared__ int marks[kWaves][kTile];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  span_sums(w, off, span, static_cast<int>(blockIdx.x) * kWaves + wave, threadIdx.x & 63,
            marks[wave], head, carry);
}

// A sequence's sums: its part in the span where it starts and the carries of
// the spans behind, G lanes (256: a workgroup).  The first lane has them.
template <int G>
__device__ __forceinline__ Sums sequence_sums(const Offsets& off, int s, int span,
                                              const Sums* head, const Sums* carry) {
  Sums sum{0.0, 0.0, 0, 0};
  const int l = threadIdx.x % G;
  if (s < off.count) {
    const int lo = off.at(s), hi = off.at(s + 1);
    if (lo < hi) {
      if (l == 0) sum = head[s];
      const int last = (hi - 1) / span;
#pragma unroll 4
      for (int k = lo / span + 1 + l; k <= last; k += G) sum.add(carry[k]);
    }
  }
  sum.template join<(G < 64 ? G : 64)>();
  if constexpr (G > 64) {
    __shared__ Sums red[G / 64];
    __syncthreads();  // (a second sequence's: the first's are read)
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
    __syncthreads();
    sum = red[0];
#pragma unroll
    for (int k = 1; k < G / 64; ++k) sum.add(red[k]);
  }
  return sum;
}

struct PolicyOut {
  float *loss, *kl;
  int32_t *count, *clipped;
  int mean;
  // of results: sequences
  __device__ __forceinline__ int results(const Offsets& off) const { return off.count; }
  template <int G>
  __device__ __forceinline__ void finish(const Offsets& off, int s, int span, const Sums* head,
                                         const Sums* carry) const {
    const Sums sum = sequence_sums<G>(off, s, span, head, carry);
    if (s >= off.count || threadIdx.x % G != 0) return;
    const double part = mean ? 1.0 / max(sum.c, 1) : 1.0;
    loss[s] = static_cast<float>(sum.a * part);
    kl[s] = static_cast<float>(sum.b * part);
    count[s] = sum.c;
    clipped[s] = sum.d;
  }
};

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
  // smoothing s(x) - (1 - smoothing) s(-x), s(x) = 1 / (1 + e^-x): e^-|x| gives
  // both s without a difference, which would lose the smaller one (smoothing - s(-x)
  // all of it with smoothing 1 and x < -17)
  const float t = expf(-fabsf(x)), big = 1.0f / (1.0f + t), small = t * big;
  return h.smoothing * (x < 0.0f ? small : big) -
         (1.0f - h.smoothing) * (x < 0.0f ? big : small);
}

struct PreferenceOut {
  float *loss, *margin, *reward;
  int32_t* count;
  PreferenceHow h;
  // of results: pairs
  __device__ __forceinline__ int results(const Offsets& off) const { return off.count / 2; }
  template <int G>
  __device__ __forceinline__ void finish(const Offsets& off, int i, int span, const Sums* head,
                                         const Sums* carry) const {
    double value[2];
    int tokens[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const Sums sum =
          sequence_sums<G>(off, i < off.count / 2 ? 2 * i + k : off.count, span, head, carry);
      value[k] = h.beta * sum.a;
      if (h.mean) value[k] /= max(sum.c, 1);
      tokens[k] = sum.c;
    }
    if (i >= off.count / 2 || threadIdx.x % G != 0) return;
    const double x = value[0] - value[1] - h.margin;
    float r = static_cast<float>(x);
    // the slope, which the backward takes from the margin, has a step at the
    // hinge's border: a margin below it stays below
    if (h.kind == MUON_PREFERENCE_HINGE && x < 1.0 && r == 1.0f) r = 1.0f - 0x1p-24f;
    margin[i] = r;
    loss[i] = tokens[0] > 0 && tokens[1] > 0 ? static_cast<float>(preference(h, x)) : 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      reward[2 * i + k] = static_cast<float>(value[k]);
      count[2 * i + k] = tokens[k];
    }
  }
};

template <int G, typename Out>
__global__ __launch_bounds__(kThreads) void k_seq_join(Offsets off, int span,
                                                       const Sums* __restrict__ head,
                                                       const Sums* __restrict__ carry, Out out) {
  out.template finish<G>(off, blockIdx.x * (kThreads / G) + threadIdx.x / G, span, head, carry);
}

// Few tokens and few sequences: the sums and their join in one workgroup, a
// tile a wave, the parts in LDS.  (Policy forward, us, this way and with two
// launches: 8192 tokens of 16 sequences 14.2 and 17.3, 16384 of 64, two tiles a
// wave, 17.2 and 17.3, 32768 29.1 and 16.8.)
constexpr int kSmallThreads = 1024, kSmallWaves = kSmallThreads / 64;
constexpr int kSmallTokens = kSmallWaves * kTile, kSmallSequences = 1024;
template <typename Terms, typename Out>
__global__ __launch_bounds__(kSmallThreads) void k_seq_small(Terms w, Offsets off,
                                                             Out out) {
  __shared__ int marks[kSmallWaves][kTile];
  __shared__ Sums head[kSmallSequences], carry[kSmallWaves];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  span_sums(w, off, kTile, wave, threadIdx.x & 63, marks[wave], head, carry);
  __syncthreads();
  constexpr int G = kSmallWaves;  // as many lanes as there can be spans
  for (int r0 = 0; r0 < out.results(off); r0 += blockDim.x / G)
    out.template finish<G>(off, r0 + threadIdx.x / G, kTile, head, carry);
}

struct PolicySlope {
  PolicyArgs p;
  const float* dloss;
  const int32_t* count;
  int mean;
  using Value = Two;  // the sequence's advantage, and its factor of a token's slope
  __device__ __forceinline__ const uint8_t* mask() const { return p.mask; }
  template <bool WHOLE>
  __device__ __forceinline__ void load(int i, int n, Tokens& t) const {
    p.load<WHOLE>(i, n, t);
  }
  __device__ __forceinline__ Value of(int s) const {
    Value v{p.per_token ? 0.0f : p.adv[s], dloss[s]};
    if (mean) v.b /= static_cast<float>(max(count[s], 1));
    return v;
  }
  __device__ __forceinline__ void slopes(const Tokens& t, int in, const Value (&v)[kPer],
                                         float (&g)[kPer]) const {
    float a[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) a[j] = p.per_token ? t.adv[j] : v[j].a;
    const int cut = p.ratios(t, a, g);
#pragma unroll
    for (int j = 0; j < kPer; ++j) g[j] = ((cut >> j) & 1) != 0 ? 0.0f : g[j] * a[j];
    if (p.kl_weight != 0.0f) {
      float em1[kPer], k[kPer];
      p.kl(t, em1, k);
#pragma unroll
      for (int j = 0; j < kPer; ++j) g[j] = __builtin_fmaf(p.kl_weight, em1[j], g[j]);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) g[j] = ((in >> j) & 1) != 0 ? v[j].b * g[j] : 0.0f;
  }
};

struct PreferenceSlope {
  const float *margin, *dloss;
  const int32_t* count;
  const uint8_t* mask_p;
  PreferenceHow h;
  using Value = One;  // a token's slope
  __device__ __forceinline__ const uint8_t* mask() const { return mask_p; }
  template <bool WHOLE>
  __device__ __forceinline__ void load(int i, int n, Tokens& t) const {
    if (mask_p != nullptr) load_values<WHOLE>(mask_p, i, n, t.mask);
  }
  __device__ __forceinline__ Value of(int s) const {
    const int i = s >> 1, mine = count[s], other = count[s ^ 1];
    const float g = h.beta * dloss[i] * preference_slope(h, margin[i]);
    if (mine <= 0 || other <= 0) return {0.0f};
    const float v = (s & 1) != 0 ? g : -g;
    return {h.mean ? v / static_cast<float>(mine) : v};
  }
  __device__ __forceinline__ void slopes(const Tokens&, int in, const Value (&v)[kPer],
                                         float (&g)[kPer]) const {
#pragma unroll
    for (int j = 0; j < kPer; ++j) g[j] = ((in >> j) & 1) != 0 ? v[j].a : 0.0f;
  }
};

// dnll of the tokens that are in a sequence.
template <typename Slope>
__global__ __launch_bounds__(kThreads) void k_seq_slopes(const Slope w, Offsets off, int span,
                                                         float* __restrict__ dnll) {
  __shared__ int marks[kWaves][kTile];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = (static_cast<int>(blockIdx.x) * kWaves + wave) * span;
  const int n = off.n, t1 = min(t0 + span, n);
  if (t0 >= n) return;
  Tokens tok;
  load_tile(w, t0, lane, n, tok);
  Walk<Slope> walk;
  walk.find(off, w, t0, lane);
  for (int tile0 = t0; tile0 < t1; tile0 += kTile) {
    const int i = tile0 + lane * kPer;
    int start[kPer], s;
    const bool any = walk.tile(off, w, tile0, lane, marks[wave], start, s);
    typename Slope::Value v[kPer];
    float g[kPer];
    const int inside = walk.values(off, w, any, s, start, v);
    w.slopes(tok, inside & counting(tok, w.mask(), i, n), v, g);
    if (tile0 + kTile < t1) load_tile(w, tile0 + kTile, lane, n, tok);
    if (inside == 0xff && i + kPer <= n) {
      __builtin_memcpy(dnll + i, g, sizeof(g));
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (((inside >> j) & 1) != 0 && i + j < n) dnll[i + j] = g[j];
    }
  }
}

// -------------------------------------------------------------------- host

// Most waves of a launch.  Spans of a few tiles: fewer, longer ones leave
// loads waiting, single tiles pay for the search and the carry each time
// (policy step of 33.5 M tokens and preference step of 16.8 M, us: 8192 spans
// 227 and 62, 16384 217 and 63, 24576 214 and 63, 32768 213 and 68, 65536 227
// and 68).
constexpr int64_t kSpans = 24576;
constexpr int64_t kFewResults = 512;
constexpr int64_t kMaxSequences = static_cast<int64_t>(1) << 24;

int span_of(int64_t n) {
  return static_cast<int>((n + kSpans * kTile - 1) / (kSpans * kTile)) * kTile;
}
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
  p.f_low = static_cast<float>(p.d_low);
  p.f_high = static_cast<float>(p.d_high);
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

template <typename Terms, typename Out>
void launch_sums(const Terms& w, const Offsets& off, int64_t results, Sums* head, Sums* carry,
                 const Out& out, hipStream_t s) {
  if (off.n <= kSmallTokens && off.count <= kSmallSequences) {
    const int waves = std::max((off.n + kTile - 1) / kTile, 4);
    hipLaunchKernelGGL((k_seq_small<Terms, Out>), dim3(1), dim3(64 * waves), 0, s, w, off, out);
    return;
  }
  const int64_t blocks = (spans_of(off.n) + kWaves - 1) / kWaves;
  if (blocks > 0)
    hipLaunchKernelGGL(k_seq_sums<Terms>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s,
                       w, off, span_of(off.n), head, carry);
  // a wave a result, or a workgroup where there are few, whose sequences can
  // have thousands of carries
  const int span = std::max(span_of(off.n), 1);
  if (results <= kFewResults)
    hipLaunchKernelGGL((k_seq_join<kThreads, Out>), dim3(static_cast<unsigned>(results)),
                       dim3(kThreads), 0, s, off, span, head, carry, out);
  else
    hipLaunchKernelGGL((k_seq_join<64, Out>),
                       dim3(static_cast<unsigned>((results + kWaves - 1) / kWaves)), dim3(kThreads),
                       0, s, off, span, head, carry, out);
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
  launch_sums(terms, off, sequences, head, carry, PolicyOut{loss, kl, count, clipped, mean != 0},
              stream);
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
  slope.p = p;
  if (kl_weight == 0.0f) slope.p.ref = nullptr;
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
  terms.nll = nll;
  terms.ref = ref_nll;
  terms.mask_p = mask;
  launch_sums(terms, off, sequences / 2, head, carry,
              PreferenceOut{loss, margins, reward, count,
                            PreferenceHow{kind, mean != 0, beta, margin, smoothing}},
              stream);
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
