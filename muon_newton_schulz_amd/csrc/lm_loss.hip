// Softmax cross entropy of a linear head over a large vocabulary, without
// keeping the logits, and its gradient.
//
//   l_tv   = h_t . W_v
//   lse_t  = log sum_v exp l_tv,   loss_t = lse_t - l_{t, y_t}
//   g_tv   = (exp(l_tv - lse_t) - [v = y_t]) dloss_t
//   dh_t   = sum_v g_tv W_v,       dW_v   = sum_t g_tv h_t        (+ dW_v)
//
// Forward: every output tile of h W^T stays in registers; a row of it leaves
// its maximum m and its sum of exp(l - m) (fp32), and the target's logit.
// A second kernel joins the tiles of a row, in order.
//
// Backward, one piece of the vocabulary after another: the piece's logits
// are computed again and turned into g / c in the epilogue, with c the
// largest |dloss|; then dW of the piece = c (g/c)^T h and dh += c (g/c) W,
// summed over the pieces in fp32.  The matrix cores take bf16, so bf16 calls
// store g / c as two bf16 planes, the nearest value (high) and what is left
// of it (low), off by 2^-16 of it at most; both products run over the low
// plane and then the high one.  One plane alone is off by up to 2^-8, and not
// at random: a row's target value, -(1 - p) dloss, is most of its gradient.
// Norm of the error of fp32 dhidden, 1024 x 32000 x 256: 1.5e-3 with random
// dloss and 3.8e-3 with two values of it, against 2.2e-6 and 4.5e-6 with two
// planes (fp32 products of the same g: 1.7e-6).  It costs the two products
// twice their work: backward of 8192 x 32000 x 2048 2.93 -> 4.84 ms, of 4096 x
// 163840 x 7168 24.7 -> 41.1 ms.  The division keeps both planes within bf16's
// range whatever the size of dloss.  Few rows give few tiles of dh with a long
// sum: it is split over workgroups, which add into fp32 sums of their own, and
// a last kernel joins those in order.
#include <algorithm>
#include <cmath>

#include "train_gemm.h"

namespace muon {
namespace {

constexpr int kThreads = 256;

// target of row t, -1 if it has none (outside [0, vocab))
__device__ __forceinline__ int64_t target_of(const void* targets, int t64, int64_t t,
                                             int64_t vocab) {
  const int64_t v = t64 ? static_cast<const int64_t*>(targets)[t]
                        : static_cast<int64_t>(static_cast<const int32_t*>(targets)[t]);
  return v >= 0 && v < vocab ? v : -1;
}

// exp: the fp32 path takes the accurate one, the bf16 path the hardware's, whose
// relative error, 2^-21 at |x| = 8, is below the 2^-16 that g keeps.  The loss
// gains nothing from the accurate one, whose terms' errors average out (rms
// error, 1024 x 32000 x 256: 5.6e-7 with it, 5.5e-7 without), and the forward of
// 8192 x 32000 x 2048 takes 940 us with it and 878 without.
template <typename T>
__device__ __forceinline__ float exp_of(float x) {
  if constexpr (sizeof(T) == 4) return expf(x);
  else return __expf(x);
}

// (m, s) <- (m, s) + (m2, s2): sums of exp(l - m) over disjoint sets.  A set
// without a value above -inf has s = 0.
__device__ __forceinline__ void join_stats(float& m, float& s, float m2, float s2) {
  const float mm = fmaxf(m, m2);
  const float a = m == mm ? s : s * expf(m - mm);
  const float b = m2 == mm ? s2 : s2 * expf(m2 - mm);
  m = mm;
  s = a + b;
}

struct StatsArgs {
  const void* h;
  const void* w;
  const void* targets;
  float* tile_m;  // [vocabulary tiles][n]
  float* tile_s;
  float* at;      // [n], the target's logit
  int64_t ldh, vocab;
  int n, dim, t64;
};

// Row statistics of one tile: the maximum and the sum of a lane's 16 NJ
// values of a row, joined with the lane that holds the row's other columns
// (lane ^ 32), then with the waves beside it.
template <typename T>
struct LossTile : TileArgs<T> {
  int i0, j0, s;
  int64_t v0;
};
template <typename Core, typename T>
__device__ __forceinline__ void stats_out(const StatsArgs& a, const LossTile<T>& w,
                                          f32x16_t (&acc)[Core::NJ][Core::MI]) {
  const int i0 = w.i0, jn = w.qn;
  const int64_t v0 = w.v0;
  const int lane = opaque_lane(), wave = threadIdx.x >> 6;
  const int wi = wave % Core::WM, wj = wave / Core::WM;
  const int jw = wj * 32 * Core::NJ + 4 * (lane >> 5);
  float* red = reinterpret_cast<float*>(Core::lds());  // [WN][BM][2]
  static_assert(Core::WN * Core::BM * 8 <= Core::kLdsBytes, "the waves' row statistics");
  // EDGE: the vocabulary ends inside the tile (the test stays out of the
  // loops of the other tiles)
  auto rows = [&](auto edge_c) {
    constexpr bool EDGE = decltype(edge_c)::value;
#pragma unroll
    for (int bi = 0; bi < Core::MI; ++bi) {
      const int i = wi * 32 * Core::MI + 32 * bi + (lane & 31);
      const int64_t t = static_cast<int64_t>(i0) + i;
      const int64_t tgt = t < a.n ? target_of(a.targets, a.t64, t, a.vocab) : -1;
      // few lanes hold their row's target
      const int64_t at64 = tgt - v0 - jw;
      const int at = tgt >= 0 && at64 >= 0 && at64 < 32 * Core::NJ ? static_cast<int>(at64) : -1;
      if (__ballot(at >= 0) != 0) {
#pragma unroll
        for (int bj = 0; bj < Core::NJ; ++bj)
#pragma unroll
          for (int v = 0; v < 16; ++v)
            if (at == 32 * bj + 8 * (v >> 2) + (v & 3)) a.at[t] = acc[bj][bi][v];
      }
      float m = -INFINITY;
#pragma unroll
      for (int bj = 0; bj < Core::NJ; ++bj)
#pragma unroll
        for (int v = 0; v < 16; ++v)
          if (!EDGE || jw + 32 * bj + 8 * (v >> 2) + (v & 3) < jn) m = fmaxf(m, acc[bj][bi][v]);
      // nothing above -inf: every term is exp(-inf) = 0
      const float ms = m == -INFINITY ? 0.0f : m;
      float s = 0.0f;
#pragma unroll
      for (int bj = 0; bj < Core::NJ; ++bj)
#pragma unroll
        for (int v = 0; v < 16; ++v)
          if (!EDGE || jw + 32 * bj + 8 * (v >> 2) + (v & 3) < jn)
            s += exp_of<T>(acc[bj][bi][v] - ms);
      const float m2 = __shfl_xor(m, 32, 64), s2 = __shfl_xor(s, 32, 64);
      if (lane < 32) {
        join_stats(m, s, m2, s2);
        red[(wj * Core::BM + i) * 2] = m;
        red[(wj * Core::BM + i) * 2 + 1] = s;
      }
      __builtin_amdgcn_sched_barrier(0);  // one block of rows at a time: fewer live values
    }
  };
  if (jn < Core::BN) rows(std::true_type{});
  else rows(std::false_type{});
  lds_barrier();
  for (int i = threadIdx.x; i < Core::BM && i0 + i < a.n; i += kThreads) {
    float m = red[2 * i], s = red[2 * i + 1];
#pragma unroll
    for (int k = 1; k < Core::WN; ++k)
      join_stats(m, s, red[(k * Core::BM + i) * 2], red[(k * Core::BM + i) * 2 + 1]);
    const int64_t o = static_cast<int64_t>(w.j0 / Core::BN) * a.n + i0 + i;
    a.tile_m[o] = m;
    a.tile_s[o] = s;
  }
}
template <typename Core, typename T>
__global__ __launch_bounds__(kThreads, Core::kWaves) void k_loss_stats(StatsArgs a, int nx, int ny) {
  using W = LossTile<T>;
  int x, y;
  if (!my_tile(nx, ny, x, y)) return;
  W w;
  w.i0 = x * Core::BM;
  w.j0 = y * Core::BN;
  w.v0 = w.j0;
  w.P = static_cast<const T*>(a.h) + w.i0 * a.ldh;
  w.ldp = a.ldh;
  w.pn = a.n - w.i0;
  w.Q = static_cast<const T*>(a.w) + w.v0 * a.dim;
  w.ldq = w.K = a.dim;
  w.qn = static_cast<int>(a.vocab - w.v0 < Core::BN ? a.vocab - w.v0 : Core::BN);
  f32x16_t acc[Core::NJ][Core::MI];
  Core::run(w, acc);
  stats_out<Core, T>(a, w, acc);
}

// Joins a row's tiles in a fixed order: thread (r, p) of a workgroup takes
// tiles p, p + P, ... of row r, R rows x P parts, then the parts are joined
// pairwise.  Rows run along the lanes, so loads of many rows are whole lines; few
// rows take more parts.
template <int R>
__global__ __launch_bounds__(kThreads) void k_loss_join(const float* __restrict__ tile_m,
                                                        const float* __restrict__ tile_s,
                                                        const float* __restrict__ at, int tiles,
                                                        int n, const void* targets, int t64,
                                                        int64_t vocab, float* __restrict__ loss,
                                                        float* __restrict__ lse) {
  constexpr int P = kThreads / R;
  __shared__ float red[kThreads / 64][R][2];
  const int r = threadIdx.x % R, part = threadIdx.x / R;
  const int t = blockIdx.x * R + r;
  float m = -INFINITY, s = 0.0f;
  if (t < n) {
    constexpr int U = 8;
    for (int k0 = part; k0 < tiles; k0 += U * P) {
      float tm[U], ts[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * P;
        tm[u] = k < tiles ? tile_m[static_cast<int64_t>(k) * n + t] : -INFINITY;
        ts[u] = k < tiles ? tile_s[static_cast<int64_t>(k) * n + t] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) join_stats(m, s, tm[u], ts[u]);
    }
  }
  // the parts of a wave, then the four waves
#pragma unroll
  for (int o = R; o < 64; o <<= 1) {
    const float m2 = __shfl_xor(m, o, 64), s2 = __shfl_xor(s, o, 64);
    join_stats(m, s, m2, s2);
  }
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) < R) {
    red[wave][r][0] = m;
    red[wave][r][1] = s;
  }
  __syncthreads();
  if (part != 0 || t >= n) return;
#pragma unroll
  for (int p = 1; p < kThreads / 64; ++p) join_stats(m, s, red[p][r][0], red[p][r][1]);
  // (m - at) + log s, not lse - at: the rounding of lse, half a step of m, is
  // all there is of a likely target's loss
  const float ls = logf(s);
  lse[t] = m + ls;
  loss[t] = target_of(targets, t64, t, vocab) >= 0 ? (m - at[t]) + ls : 0.0f;
}

// c: the largest finite |dloss| of the rows with a target, 1 if that is 0.
constexpr int kScaleThreads = 1024;
__global__ __launch_bounds__(kScaleThreads) void k_loss_scale(const float* __restrict__ dloss, int n,
                                                              const void* targets, int t64,
                                                              int64_t vocab, float* c) {
  __shared__ float red[kScaleThreads / 64];
  float m = 0.0f;
  for (int t = threadIdx.x; t < n; t += kScaleThreads) {
    const float a = fabsf(dloss[t]);
    if (a < INFINITY && target_of(targets, t64, t, vocab) >= 0) m = fmaxf(m, a);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int k = 1; k < kScaleThreads / 64; ++k) m = fmaxf(m, red[k]);
  *c = m > 0.0f ? m : 1.0f;
}

struct GradArgs {
  const void* h;
  const void* w;       // the piece's first row
  const void* targets;
  const float* lse;
  const float* dloss;
  const float* c;
  void* g;             // [n][ldg], g / c; bf16: low plane, high plane
  int64_t ldh, ldg, vocab, v0;
  int n, dim, len, t64;  // len: vocabulary rows of the piece
};

// What rounding to bf16 leaves of each value (0 where that is not finite).
template <int NJ, int MI>
__device__ __forceinline__ void low_part(f32x16_t (&acc)[NJ][MI]) {
#pragma unroll
  for (int a = 0; a < NJ; ++a)
#pragma unroll
    for (int b = 0; b < MI; ++b)
#pragma unroll
      for (int v = 0; v < 16; v += 2) {
        const uint32_t h = pack_bf16(acc[a][b][v], acc[a][b][v + 1]);
        const float x = acc[a][b][v] - __uint_as_float(h << 16);
        const float y = acc[a][b][v + 1] - __uint_as_float(h & 0xffff0000u);
        acc[a][b][v] = fabsf(x) < INFINITY ? x : 0.0f;
        acc[a][b][v + 1] = fabsf(y) < INFINITY ? y : 0.0f;
      }
}

// g / c of the piece, in the operands' type (bf16: two planes).
template <typename Core, typename T>
__device__ __forceinline__ void g_out(const GradArgs& a, const LossTile<T>& w,
                                      f32x16_t (&acc)[Core::NJ][Core::MI]) {
  const int i0 = w.i0, j0 = w.j0;
  const int lane = opaque_lane(), wave = threadIdx.x >> 6;
  const int iw = (wave % Core::WM) * 32 * Core::MI + (lane & 31);
  float lse[Core::MI], dl[Core::MI];
  int64_t tgt[Core::MI];
#pragma unroll
  for (int bi = 0; bi < Core::MI; ++bi) {
    const int64_t t = static_cast<int64_t>(i0) + iw + 32 * bi;
    lse[bi] = dl[bi] = 0.0f;
    tgt[bi] = -1;
    if (t < a.n) {
      tgt[bi] = target_of(a.targets, a.t64, t, a.vocab);
      lse[bi] = a.lse[t];
      dl[bi] = a.dloss[t] / *a.c;
    }
  }
  // A row without a target has no loss, whatever dloss holds there.  On the
  // grid the columns from the piece's end to ldg are stored as zeros, which
  // the sums over the vocabulary read.
  const int jw = (wave / Core::WM) * 32 * Core::NJ + 4 * (lane >> 5);
  const int len = a.len - j0 - jw;
#pragma unroll
  for (int bi = 0; bi < Core::MI; ++bi) {
    const bool row = tgt[bi] >= 0;
    const int64_t at64 = tgt[bi] - a.v0 - j0 - jw;
    const int at = row && at64 >= 0 && at64 < 32 * Core::NJ ? static_cast<int>(at64) : -1;
    const int left = row ? len : 0;
#pragma unroll
    for (int bj = 0; bj < Core::NJ; ++bj)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int j = 32 * bj + 8 * (v >> 2) + (v & 3);
        const float p = exp_of<T>(acc[bj][bi][v] - lse[bi]);
        acc[bj][bi][v] = j < left ? (at == j ? p - 1.0f : p) * dl[bi] : 0.0f;
      }
    __builtin_amdgcn_sched_barrier(0);
  }
  T* low = static_cast<T*>(a.g) + i0 * a.ldg + j0;
  const int cols = Core::kGrid ? static_cast<int>(a.ldg) - j0 : a.len - j0;
  const T* none = nullptr;
  if constexpr (sizeof(T) == 2) {
    Core::write(acc, low + a.n * a.ldg, a.ldg, none, 0, a.n - i0, cols);
    low_part(acc);
  }
  Core::write(acc, low, a.ldg, none, 0, a.n - i0, cols);
}

// A product with g: the sum over its planes, `plane` elements apart.
template <typename Core, typename T>
__device__ __forceinline__ void run_planes(LossTile<T>& w, int64_t plane,
                                           f32x16_t (&acc)[Core::NJ][Core::MI]) {
  if constexpr (sizeof(T) == 2) {
    zero_acc(acc);
#pragma unroll 1
    for (int p = 0; p < 2; ++p, w.P += plane) Core::template run<true>(w, acc);
  } else {
    Core::run(w, acc);
  }
}

template <typename Core, typename T>
__global__ __launch_bounds__(kThreads, Core::kWaves) void k_loss_g(GradArgs a, int nx, int ny) {
  using W = LossTile<T>;
  int x, y;
  if (!my_tile(nx, ny, x, y)) return;
  W w;
  w.i0 = x * Core::BM;
  w.j0 = y * Core::BN;
  w.P = static_cast<const T*>(a.h) + w.i0 * a.ldh;
  w.ldp = a.ldh;
  w.pn = a.n - w.i0;
  w.Q = static_cast<const T*>(a.w) + static_cast<int64_t>(w.j0) * a.dim;
  w.ldq = w.K = a.dim;
  w.qn = a.len - w.j0;
  f32x16_t acc[Core::NJ][Core::MI];
  Core::run(w, acc);
  g_out<Core, T>(a, w, acc);
}

// hidden with zeros in the rows without a target, [n][dim]: dW's sum runs over
// all rows, and 0 times what such a row holds is 0 only where that is finite.
// One read and one write of hidden (backward of 8192 x 32000 x 2048: 4.60 ms
// against 4.56 without, of 33 x 32000 x 2048: 114 us against 112).
template <typename T>
__global__ __launch_bounds__(kThreads) void k_loss_rows(const T* __restrict__ h, int64_t ldh,
                                                        const void* targets, int t64, int n,
                                                        int dim, int64_t vocab,
                                                        T* __restrict__ out) {
  constexpr int E = 16 / sizeof(T);
  const int per = (dim + E - 1) / E;
  const int64_t total = static_cast<int64_t>(n) * per;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t t = i / per;
    const int c = static_cast<int>(i - t * per) * E;
    const bool row = target_of(targets, t64, t, vocab) >= 0;
    const T* p = h + t * ldh + c;
    T* o = out + t * dim + c;
    if (c + E <= dim) {
      u32x4_t v = {0, 0, 0, 0};
      if (row) __builtin_memcpy(&v, p, 16);
      __builtin_memcpy(o, &v, 16);
    } else {
      for (int e = 0; c + e < dim; ++e) o[e] = row ? p[e] : T{};
    }
  }
}

struct DhArgs {
  const void* g;
  const void* w;  // the piece's first row
  const void* targets;
  const float* c;
  float* part;    // fp32 sums, [splits][n][dim]
  void* out;      // dhidden, or null: leave the sums in part
  int64_t ldg, ld_out, vocab;
  int n, dim, len, splits, first, t64;
};

// dh (+)= g W of the piece; split s takes its share of the piece's rows.
template <typename Core, typename T, typename TO>
__global__ __launch_bounds__(kThreads, Core::kWaves) void k_loss_dh(DhArgs a, int nx, int ny) {
  using W = LossTile<T>;
  // shares in whole steps of 64 rows
  const int share = ((a.len + a.splits - 1) / a.splits + 63) / 64 * 64;
  int x, y;
  if (!my_tile(nx, static_cast<int64_t>(ny) * a.splits, x, y)) return;
  W w;
  w.s = y / ny;
  w.i0 = x * Core::BM;
  w.j0 = y % ny * Core::BN;
  const int k0 = min(w.s * share, a.len);
  w.P = static_cast<const T*>(a.g) + w.i0 * a.ldg + k0;
  w.ldp = a.ldg;
  w.pn = a.n - w.i0;
  w.Q = static_cast<const T*>(a.w) + static_cast<int64_t>(k0) * a.dim + w.j0;
  w.ldq = a.dim;
  w.qn = a.dim - w.j0;
  w.K = min(share, a.len - k0);
  f32x16_t acc[Core::NJ][Core::MI];
  run_planes<Core, T>(w, a.n * a.ldg, acc);
  // no gradient for a row without a target, where a weight is not finite too
  const float c = *a.c;
  const int t0 = w.i0 + (threadIdx.x >> 6) % Core::WM * 32 * Core::MI + (opaque_lane() & 31);
#pragma unroll
  for (int bi = 0; bi < Core::MI; ++bi) {
    const int t = t0 + 32 * bi;
    const bool row = t < a.n && target_of(a.targets, a.t64, t, a.vocab) >= 0;
#pragma unroll
    for (int bj = 0; bj < Core::NJ; ++bj)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[bj][bi][v] = row ? acc[bj][bi][v] * c : 0.0f;
  }
  float* D = a.part + (static_cast<int64_t>(w.s) * a.n + w.i0) * a.dim + w.j0;
  const float* old = a.first ? nullptr : D;
  if (a.out == nullptr)
    Core::write(acc, D, a.dim, old, a.dim, w.pn, w.qn);
  else
    Core::write(acc, static_cast<TO*>(a.out) + w.i0 * a.ld_out + w.j0, a.ld_out, old, a.dim,
                w.pn, w.qn);
}

// dhidden = sum of the splits, in order.
template <typename TO>
__global__ __launch_bounds__(kThreads) void k_loss_dh_join(const float* __restrict__ part,
                                                           int splits, int n, int dim, TO* out,
                                                           int64_t ld) {
  const int64_t total = static_cast<int64_t>(n) * dim;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    float v = part[i];
    for (int s = 1; s < splits; ++s) v += part[s * total + i];
    from_f32(v, out + i / dim * ld + i % dim);
  }
}

struct DwArgs {
  const void* g;
  const void* h;  // k_loss_rows' copy
  const float* c;
  void* dw;  // the piece's first row
  int64_t ldg, ldh, vocab;
  int n, dim, len, accumulate;
};

template <typename Core, bool STREAM, typename T, typename TO>
__global__ __launch_bounds__(kThreads, Core::kWaves) void k_loss_dw(DwArgs a, int nx, int ny) {
  using W = LossTile<T>;
  int x, y;
  if (!my_tile(nx, ny, x, y)) return;
  W w;
  w.i0 = x * Core::BM;
  w.j0 = y * Core::BN;
  w.P = static_cast<const T*>(a.g) + w.i0;
  w.ldp = a.ldg;
  w.pn = a.len - w.i0;
  w.Q = static_cast<const T*>(a.h) + w.j0;
  w.ldq = a.ldh;
  w.qn = a.dim - w.j0;
  w.K = a.n;
  f32x16_t acc[Core::NJ][Core::MI];
  run_planes<Core, T>(w, a.n * a.ldg, acc);
  scale_acc(acc, *a.c);
  TO* C = static_cast<TO*>(a.dw) + static_cast<int64_t>(w.i0) * a.dim + w.j0;
  Core::template write<STREAM>(acc, C, a.dim, a.accumulate ? C : static_cast<const TO*>(nullptr),
                               a.dim, w.pn, w.qn);
}

template <typename T>
__global__ void k_zero_rows(T* p, int64_t rows, int64_t cols, int64_t ld) {
  const int64_t total = rows * cols;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x)
    p[i / cols * ld + i % cols] = T{};
}

// -------------------------------------------------------------------- host

constexpr int kTile = 64;  // the narrowest tile: bounds the tile statistics
// Forward: rows per pass, which bounds the tile statistics (vocab / 16 bytes
// a row) without leaving the GPU short of tiles.
constexpr int64_t kStatsRows = 16384;
// Backward: bytes of a plane of g at a time.  Fewer pieces mean fewer passes
// over the fp32 sums of dh; g should stay near what the last-level cache holds
// (bf16, two planes, 8192 x 32000 x 2048: 4.84 ms, with half of it 5.00; 4096 x
// 163840 x 7168: 41.1 and 42.2).
constexpr int64_t kPieceBytes = static_cast<int64_t>(256) << 20;
constexpr int64_t kMinPiece = 2048, kPieceStep = 256;  // whole tiles
// A launch holds fewer than 2^24 workgroups of 256: kStatsRows x kMaxVocabLoss
// and kMaxTokensLoss x kMinPiece in 64 x 64 tiles are at most 2^23.
constexpr int64_t kMaxVocabLoss = static_cast<int64_t>(1) << 21;
constexpr int64_t kMaxTokensLoss = static_cast<int64_t>(1) << 24;
// Shares of dh's sum at most: the tiles of the core for any operands take
// longer, and gain from more (backward of 515 x 33001 x 500: fp32 507 us with
// 16, 455 with 25; bf16 342 and 285; DMA core, 33 x 32000 x 2048: 112 and, with
// 32, 119).
constexpr int kMaxSplits = 16, kMaxSplitsAny = 32;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
auto row_tiles(int64_t rows) {
  return [rows](int bm) { return static_cast<double>(ceil_div(rows, bm)); };
}
// dh: `splits` times the tiles, each with its share of the sum
auto dh_tiles(int64_t n, int splits) {
  return [n, splits](int bm) { return static_cast<double>(ceil_div(n, bm) * splits); };
}

struct LossWs {
  int64_t stats_rows, v_tiles;          // forward
  int64_t piece, ldg;                   // backward
  int splits;
  size_t tile_m, tile_s, at, c, g, rows, part, total;
};
LossWs loss_ws(int64_t n, int64_t vocab, int64_t dim, int32_t dtype, bool backward) {
  LossWs w{};
  size_t o = 0;
  // forward
  w.stats_rows = std::min(n, kStatsRows);
  w.v_tiles = ceil_div(vocab, kTile);
  w.tile_m = o;
  o += align256(static_cast<size_t>(w.stats_rows * w.v_tiles) * 4);
  w.tile_s = o;
  o += align256(static_cast<size_t>(w.stats_rows * w.v_tiles) * 4);
  w.at = o;
  o += align256(static_cast<size_t>(w.stats_rows) * 4);
  w.total = o;
  if (!backward) return w;
  // backward (the forward's part of the workspace is free again)
  o = 0;
  const int64_t sz = static_cast<int64_t>(train_dtype_size(dtype));
  const int64_t planes = dtype == MUON_DTYPE_BF16 ? 2 : 1;
  w.piece = std::max(kMinPiece, kPieceBytes / (sz * n) / kPieceStep * kPieceStep);
  if (w.piece >= vocab) {
    w.piece = vocab;
  } else {
    // pieces of equal length, whole tiles
    const int64_t pieces = ceil_div(vocab, w.piece);
    w.piece = ceil_div(ceil_div(vocab, pieces), kPieceStep) * kPieceStep;
  }
  // off the multiples of 4 KiB, where the rows of a tile fall on the same
  // memory channels (backward of 4096 x 163840 x 7168: 38.7 ms against 40.6)
  w.ldg = ceil_div(w.piece, 8) * 8;
  if (w.ldg % 1024 == 0) w.ldg += 128;
  w.c = o;
  o += 256;
  w.g = o;
  o += align256(static_cast<size_t>(planes * n * w.ldg * sz));
  w.rows = o;
  o += align256(static_cast<size_t>(n * dim * sz));
  // dh tiles against the GPU's 256 workgroups of one tile each
  const int64_t tiles = ceil_div(n, 128) * ceil_div(dim, 128);
  w.splits = static_cast<int>(
      std::max<int64_t>(1, std::min<int64_t>({dtype == MUON_DTYPE_BF16 && dim % 8 == 0 ? kMaxSplits : kMaxSplitsAny,
                                              512 / tiles, ceil_div(w.piece, 512)})));
  w.part = o;
  if (w.splits > 1 || w.piece < vocab)
    o += align256(static_cast<size_t>(w.splits) * static_cast<size_t>(n * dim) * 4);
  w.total = std::max(w.total, o);
  return w;
}

// bf16 operands on the 16-byte grid take the DMA core (grid), others the
// core for any operands.
template <typename Core, typename T>
int launch_stats(const StatsArgs& a, hipStream_t s) {
  const int nx = static_cast<int>(ceil_div(a.n, Core::BM));
  const int ny = static_cast<int>(ceil_div(a.vocab, Core::BN));
  hipLaunchKernelGGL((k_loss_stats<Core, T>), dim3(tile_blocks(nx, ny)),
                     dim3(kThreads), 0, s, a, nx, ny);
  return ny;
}
// returns the number of tiles along the vocabulary
template <typename T>
int run_stats(const StatsArgs& a, bool grid, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (grid) {
      const Shape shape = pick_shape(kShapeNT, row_tiles(a.n), a.vocab, a.dim);
      if (shape == kLarge) return launch_stats<LargeCore<false, false>, T>(a, s);
      if (shape == kHalf) return launch_stats<HalfCore<false, false>, T>(a, s);
      if (shape == kMedium) return launch_stats<MediumCore<false, false>, T>(a, s);
      return launch_stats<ThinCore<false, false>, T>(a, s);
    }
  }
  if (pick_any_large<T>(row_tiles(a.n), a.vocab, a.dim))
    return launch_stats<OtherCore<T, false, false, 128>, T>(a, s);
  return launch_stats<OtherCore<T, false, false, 64>, T>(a, s);
}

template <typename Core, typename T>
void launch_g(const GradArgs& a, hipStream_t s) {
  const int nx = static_cast<int>(ceil_div(a.n, Core::BM));
  const int ny = static_cast<int>(ceil_div(a.len, Core::BN));
  hipLaunchKernelGGL((k_loss_g<Core, T>), dim3(tile_blocks(nx, ny)),
                     dim3(kThreads), 0, s, a, nx, ny);
}
template <typename T>
void run_g(const GradArgs& a, bool grid, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (grid) {
      const Shape shape = pick_shape(kShapeNT, row_tiles(a.n), a.len, a.dim);
      if (shape == kLarge) return launch_g<LargeCore<false, false>, T>(a, s);
      if (shape == kHalf) return launch_g<HalfCore<false, false>, T>(a, s);
      if (shape == kMedium) return launch_g<MediumCore<false, false>, T>(a, s);
      return launch_g<ThinCore<false, false>, T>(a, s);
    }
  }
  if (pick_any_large<T>(row_tiles(a.n), a.len, a.dim))
    launch_g<OtherCore<T, false, false, 128>, T>(a, s);
  else
    launch_g<OtherCore<T, false, false, 64>, T>(a, s);
}

template <typename Core, typename T, typename TO>
void launch_dh(const DhArgs& a, hipStream_t s) {
  const int nx = static_cast<int>(ceil_div(a.n, Core::BM));
  const int ny = static_cast<int>(ceil_div(a.dim, Core::BN));
  hipLaunchKernelGGL((k_loss_dh<Core, T, TO>),
                     dim3(tile_blocks(nx, static_cast<int64_t>(ny) * a.splits)),
                     dim3(kThreads), 0, s, a, nx, ny);
}
// bf16: a sum runs over both planes of g
template <typename T>
constexpr int64_t kPlanes = sizeof(T) == 2 ? 2 : 1;
template <typename T, typename TO>
void run_dh(const DhArgs& a, bool grid, hipStream_t s) {
  const int64_t k = kPlanes<T> * ceil_div(a.len, a.splits);
  if constexpr (sizeof(T) == 2) {
    if (grid) {
      const Shape shape = pick_shape(kShapeNN, dh_tiles(a.n, a.splits), a.dim, k);
      if (shape == kLarge) return launch_dh<LargeCore<false, true>, T, TO>(a, s);
      if (shape == kHalf) return launch_dh<HalfCore<false, true>, T, TO>(a, s);
      if (shape == kMedium) return launch_dh<MediumCore<false, true>, T, TO>(a, s);
      return launch_dh<ThinCore<false, true>, T, TO>(a, s);
    }
  }
  if (pick_any_large<T>(dh_tiles(a.n, a.splits), a.dim, k))
    launch_dh<OtherCore<T, false, true, 128>, T, TO>(a, s);
  else
    launch_dh<OtherCore<T, false, true, 64>, T, TO>(a, s);
}

template <typename Core, typename T, typename TO>
void launch_dw(const DwArgs& a, hipStream_t s) {
  const int nx = static_cast<int>(ceil_div(a.len, Core::BM));
  const int ny = static_cast<int>(ceil_div(a.dim, Core::BN));
  auto* kernel = k_loss_dw<Core, false, T, TO>;
  if constexpr (Core::kGrid) {
    if (stream_gradient(static_cast<const TO*>(a.dw), a.vocab, a.dim))
      kernel = k_loss_dw<Core, true, T, TO>;
  }
  hipLaunchKernelGGL(kernel, dim3(tile_blocks(nx, ny)), dim3(kThreads), 0, s, a, nx, ny);
}
template <typename T, typename TO>
void run_dw(const DwArgs& a, bool grid, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (grid) {
      const Shape shape = pick_shape(kShapeTN, row_tiles(a.len), a.dim, kPlanes<T> * a.n);
      if (shape == kLarge) return launch_dw<LargeCore<true, true>, T, TO>(a, s);
      if (shape == kHalf) return launch_dw<HalfCore<true, true>, T, TO>(a, s);
      return launch_dw<MediumCore<true, true>, T, TO>(a, s);
    }
  }
  if (pick_any_large<T>(row_tiles(a.len), a.dim, kPlanes<T> * a.n))
    launch_dw<OtherCore<T, true, true, 128>, T, TO>(a, s);
  else
    launch_dw<OtherCore<T, true, true, 64>, T, TO>(a, s);
}

struct BackwardArgs {
  const void *h, *w, *targets;
  const float *lse, *dloss;
  void *dh, *dw;
  int64_t n, vocab, dim, ldh, ld_dh;
  int t64, accumulate;
  char* ws;
};

template <typename T, typename TH, typename TW>
void run_backward(const BackwardArgs& b, const LossWs& w, hipStream_t s) {
  T* g = reinterpret_cast<T*>(b.ws + w.g);
  float* part = reinterpret_cast<float*>(b.ws + w.part);
  float* c = reinterpret_cast<float*>(b.ws + w.c);
  hipLaunchKernelGGL(k_loss_scale, dim3(1), dim3(kScaleThreads), 0, s, b.dloss,
                     static_cast<int>(b.n), b.targets, b.t64, b.vocab, c);
  T* rows = reinterpret_cast<T*>(b.ws + w.rows);
  if (b.dw != nullptr) {
    const int64_t pieces = b.n * ceil_div(b.dim, 16 / static_cast<int64_t>(sizeof(T)));
    hipLaunchKernelGGL(k_loss_rows<T>,
                       dim3(static_cast<unsigned>(std::min<int64_t>(8192, ceil_div(pieces, kThreads)))),
                       dim3(kThreads), 0, s, static_cast<const T*>(b.h), b.ldh, b.targets, b.t64,
                       static_cast<int>(b.n), static_cast<int>(b.dim), b.vocab, rows);
  }
  const bool grid = on_grid(b.h, b.ldh, b.dim) && on_grid(b.w, b.dim, b.dim);
  for (int64_t v0 = 0; v0 < b.vocab; v0 += w.piece) {
    const int len = static_cast<int>(std::min(w.piece, b.vocab - v0));
    const T* wp = static_cast<const T*>(b.w) + v0 * b.dim;
    run_g<T>(GradArgs{b.h, wp, b.targets, b.lse, b.dloss, c, g, b.ldh, w.ldg, b.vocab, v0,
                      static_cast<int>(b.n), static_cast<int>(b.dim), len, b.t64},
             grid, s);
    if (b.dh != nullptr) {
      const bool last = v0 + len == b.vocab;
      run_dh<T, TH>(DhArgs{g, wp, b.targets, c, part, last && w.splits == 1 ? b.dh : nullptr,
                           w.ldg, b.ld_dh, b.vocab, static_cast<int>(b.n),
                           static_cast<int>(b.dim), len, w.splits, v0 == 0 ? 1 : 0, b.t64},
                    grid && on_grid(b.dh, b.ld_dh, b.dim), s);
    }
    if (b.dw != nullptr)
      run_dw<T, TW>(DwArgs{g, rows, c, static_cast<TW*>(b.dw) + v0 * b.dim, w.ldg, b.dim, b.vocab,
                           static_cast<int>(b.n), static_cast<int>(b.dim), len, b.accumulate},
                    grid && on_grid(b.dw, b.dim, b.dim), s);
  }
  if (b.dh != nullptr && w.splits > 1)
    hipLaunchKernelGGL(k_loss_dh_join<TH>,
                       dim3(static_cast<unsigned>(std::min<int64_t>(4096, ceil_div(b.n * b.dim, kThreads)))),
                       dim3(kThreads), 0, s, part, w.splits, static_cast<int>(b.n),
                       static_cast<int>(b.dim), static_cast<TH*>(b.dh), b.ld_dh);
}

int check_loss(int64_t n, int64_t vocab, int64_t dim, int64_t ldh, int32_t dtype) {
  const int rc = check_token_sizes(n, vocab, dim);
  if (rc != MUON_OK) return rc;
  if (vocab > kMaxVocabLoss)
    return set_error(MUON_ERR_UNSUPPORTED, "vocab must be at most 2^21");
  if (n > kMaxTokensLoss) return set_error(MUON_ERR_UNSUPPORTED, "n must be at most 2^24");
  if (!train_dtype_ok(dtype))
    return set_error(MUON_ERR_BAD_DTYPE, "hidden and weight must be fp32 or bf16");
  if (ldh < dim) return set_error(MUON_ERR_BAD_SHAPE, "ld_hidden < dim");
  return MUON_OK;
}

int check_ws(const void* ws, size_t bytes, size_t need, const char* who) {
  if (ws == nullptr || bytes < need || reinterpret_cast<uintptr_t>(ws) % 256 != 0)
    return set_error(MUON_ERR_WORKSPACE_TOO_SMALL, std::string(who) + " needs " +
                                                       std::to_string(need) +
                                                       " bytes of workspace, 256-byte aligned");
  return MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

size_t lm_loss_workspace_size(int64_t n, int64_t vocab, int64_t dim, int32_t dtype,
                              int32_t backward) {
  if (n <= 0 || check_loss(n, vocab, dim, dim, dtype) != MUON_OK) return 0;
  return loss_ws(n, vocab, dim, dtype, backward != 0).total;
}

int lm_loss_forward(const void* hidden, int64_t ld_hidden, const void* weight, int32_t dtype,
                    const void* targets, int32_t targets_64, int64_t n, int64_t vocab,
                    int64_t dim, float* loss, float* lse, void* workspace,
                    size_t workspace_bytes, hipStream_t stream) {
  int rc = check_loss(n, vocab, dim, ld_hidden, dtype);
  if (rc != MUON_OK) return rc;
  if (n == 0) return MUON_OK;
  if (hidden == nullptr || weight == nullptr || targets == nullptr || loss == nullptr ||
      lse == nullptr)
    return set_error(MUON_ERR_INVALID_ARG, "hidden, weight, targets, loss or lse is null");
  const LossWs w = loss_ws(n, vocab, dim, dtype, false);
  if ((rc = check_ws(workspace, workspace_bytes, w.total, "lm_loss_forward")) != MUON_OK) return rc;
  char* ws = static_cast<char*>(workspace);
  float* tm = reinterpret_cast<float*>(ws + w.tile_m);
  float* ts = reinterpret_cast<float*>(ws + w.tile_s);
  float* at = reinterpret_cast<float*>(ws + w.at);
  const size_t sz = train_dtype_size(dtype), tsz = targets_64 ? 8 : 4;
  for (int64_t r0 = 0; r0 < n; r0 += w.stats_rows) {
    const int rows = static_cast<int>(std::min(w.stats_rows, n - r0));
    const void* tg = static_cast<const char*>(targets) + static_cast<size_t>(r0) * tsz;
    const StatsArgs a{static_cast<const char*>(hidden) + static_cast<size_t>(r0 * ld_hidden) * sz,
                      weight, tg, tm, ts, at, ld_hidden, vocab, rows, static_cast<int>(dim),
                      targets_64 != 0};
    const bool grid = on_grid(a.h, ld_hidden, dim) && on_grid(weight, dim, dim);
    const int v_tiles = static_cast<int>(dtype == MUON_DTYPE_BF16 ? run_stats<uint16_t>(a, grid, stream)
                                                                 : run_stats<float>(a, grid, stream));
    // 16 rows a workgroup and 16 parts of a row; few rows take 4 and 64 (the
    // call: 33 x 32000 x 2048 27.1 us against 29.7, 512 x 163840 x 64 40.1
    // against 40.5, but 2048 x 32000 x 64 34.6 against 30.8)
    const int per = rows <= 512 ? 4 : 16;
    hipLaunchKernelGGL(per == 4 ? k_loss_join<4> : k_loss_join<16>,
                       dim3(static_cast<unsigned>(ceil_div(rows, per))), dim3(kThreads), 0, stream,
                       tm, ts, at, v_tiles, rows, tg, targets_64 != 0, vocab, loss + r0, lse + r0);
  }
  return check_launch("vocabulary loss launch");
}

int lm_loss_backward(const void* hidden, int64_t ld_hidden, const void* weight, int32_t dtype,
                     const void* targets, int32_t targets_64, int64_t n, int64_t vocab,
                     int64_t dim, const float* lse, const float* dloss, void* dhidden,
                     int32_t dhidden_dtype, int64_t ld_dhidden, void* dweight,
                     int32_t dweight_dtype, int32_t accumulate, void* workspace,
                     size_t workspace_bytes, hipStream_t stream) {
  int rc = check_loss(n, vocab, dim, ld_hidden, dtype);
  if (rc != MUON_OK) return rc;
  if (dhidden != nullptr) {
    if (!train_dtype_ok(dhidden_dtype))
      return set_error(MUON_ERR_BAD_DTYPE, "dhidden must be fp32 or bf16");
    if (ld_dhidden < dim) return set_error(MUON_ERR_BAD_SHAPE, "ld_dhidden < dim");
  }
  if (dweight != nullptr && !train_dtype_ok(dweight_dtype))
    return set_error(MUON_ERR_BAD_DTYPE, "dweight must be fp32 or bf16");
  if (n == 0) {
    // no rows: dweight is a sum of nothing
    if (dweight != nullptr && !accumulate) {
      if (dweight_dtype == MUON_DTYPE_BF16)
        hipLaunchKernelGGL(k_zero_rows<uint16_t>, dim3(4096), dim3(kThreads), 0, stream,
                           static_cast<uint16_t*>(dweight), vocab, dim, dim);
      else
        hipLaunchKernelGGL(k_zero_rows<float>, dim3(4096), dim3(kThreads), 0, stream,
                           static_cast<float*>(dweight), vocab, dim, dim);
      return check_launch("vocabulary loss gradient launch");
    }
    return MUON_OK;
  }
  if (dhidden == nullptr && dweight == nullptr) return MUON_OK;
  if (hidden == nullptr || weight == nullptr || targets == nullptr || lse == nullptr ||
      dloss == nullptr)
    return set_error(MUON_ERR_INVALID_ARG, "hidden, weight, targets, lse or dloss is null");
  const LossWs w = loss_ws(n, vocab, dim, dtype, true);
  if ((rc = check_ws(workspace, workspace_bytes, w.total, "lm_loss_backward")) != MUON_OK) return rc;
  const BackwardArgs b{hidden, weight, targets, lse, dloss, dhidden, dweight, n, vocab, dim,
                       ld_hidden, ld_dhidden, targets_64 != 0, accumulate != 0,
                       static_cast<char*>(workspace)};
  const bool hb = dhidden_dtype == MUON_DTYPE_BF16, wb = dweight_dtype == MUON_DTYPE_BF16;
#define MUON_LOSS_BWD(T)                                           \
  do {                                                             \
    if (hb && wb) run_backward<T, uint16_t, uint16_t>(b, w, stream); \
    else if (hb) run_backward<T, uint16_t, float>(b, w, stream);   \
    else if (wb) run_backward<T, float, uint16_t>(b, w, stream);   \
    else run_backward<T, float, float>(b, w, stream);              \
  } while (0)
  if (dtype == MUON_DTYPE_BF16) MUON_LOSS_BWD(uint16_t);
  else MUON_LOSS_BWD(float);
#undef MUON_LOSS_BWD
  return check_launch("vocabulary loss gradient launch");
}

}  // extern "C"
