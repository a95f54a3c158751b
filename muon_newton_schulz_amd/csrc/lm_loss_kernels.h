// The kernels behind the losses of a linear head over a large vocabulary that
// differ between them, and the choice of their tile cores: row statistics of the
// logits' tiles, and the two products with g.  Included by the cross entropy
// (lm_loss.hip, where the formulas and the kernels that do not differ stand) and,
// LISTS, by the distillation loss (distill.hip), which also takes listed columns'
// logits from the statistics' tiles.
#pragma once

#include <algorithm>
#include <cmath>

#include "lm_loss.h"
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

// Row statistics of one tile: the maximum and the sum of a lane's 16 NJ
// values of a row, joined with the lane that holds the row's other columns
// (lane ^ 32), then with the waves beside it.  LISTS: also the logits of the
// row's listed columns.
template <typename T>
struct LossTile : TileArgs<T> {
  int i0, j0, s;
  int64_t v0;
};
template <bool LISTS, typename Core, typename T>
__device__ __forceinline__ void stats_out(const StatsArgs& a, const LossTile<T>& w,
                                          f32x16_t (&acc)[Core::NJ][Core::MI]) {
  const int i0 = w.i0, jn = w.qn;
  const int64_t v0 = w.v0;
  const int lane = opaque_lane(), wave = threadIdx.x >> 6;
  const int wi = wave % Core::WM, wj = wave / Core::WM;
  const int jw = wj * 32 * Core::NJ + 4 * (lane >> 5);
  float* red = reinterpret_cast<float*>(Core::lds());  // [WN][BM][2]
  static_assert(Core::WN * Core::BM * 8 <= Core::kLdsBytes, "the waves' row statistics");
  const float scale = a.scale;
  // LISTS: the wave's columns as keys, and where each row's list reaches them
  const int64_t c0 = v0 + wj * 32 * Core::NJ;
  const uint32_t key0 = static_cast<uint32_t>(c0) << kPlaceBits;
  const uint32_t key1 = static_cast<uint32_t>(c0 + 32 * Core::NJ) << kPlaceBits;
  int first[Core::MI];
  if constexpr (LISTS) {
#pragma unroll
    for (int bi = 0; bi < Core::MI; ++bi) {
      const int64_t t = static_cast<int64_t>(i0) + wi * 32 * Core::MI + 32 * bi + (lane & 31);
      int lo = 0, len = t < a.n ? a.top : 0;
      if (len == 0) lo = a.top;
      while (len > 0) {
        const int half = len >> 1;
        if (a.keys[t * a.top + lo + half] < key0) {
          lo += half + 1;
          len -= half + 1;
        } else {
          len = half;
        }
      }
      first[bi] = lo;
    }
  }
  // EDGE: the vocabulary ends inside the tile (the test stays out of the
  // loops of the other tiles)
  auto rows = [&](auto edge_c) {
    constexpr bool EDGE = decltype(edge_c)::value;
#pragma unroll
    for (int bi = 0; bi < Core::MI; ++bi) {
      const int i = wi * 32 * Core::MI + 32 * bi + (lane & 31);
      const int64_t t = static_cast<int64_t>(i0) + i;
      if constexpr (LISTS) {
        // one entry of each lane's row at a time; the lane of the pair that
        // holds the column picks its value by the bits of the column
        for (int p = first[bi];; ++p) {
          const uint32_t key = p < a.top ? a.keys[t * a.top + p] : ~0u;
          const bool more = key < key1;
          if (__ballot(more) == 0) break;
          const int col = static_cast<int>((key - key0) >> kPlaceBits) & (32 * Core::NJ - 1);
          float x[16];
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            x[v] = acc[0][bi][v];
#pragma unroll
            for (int bj = 1; bj < Core::NJ; ++bj) x[v] = col >> 5 == bj ? acc[bj][bi][v] : x[v];
          }
          // column bits 0, 1, 3, 4 are the index's
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const bool odd = (col >> (b < 2 ? b : b + 1)) & 1;
#pragma unroll
            for (int v = 0; v < 8 >> b; ++v) x[v] = odd ? x[2 * v + 1] : x[2 * v];
          }
          if (more && ((col >> 2) & 1) == lane >> 5)
            a.points[t * a.top + (key & ((1u << kPlaceBits) - 1))] = x[0];
          if (!more) p = a.top;
        }
      } else {
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
      }
      float m = -INFINITY;
#pragma unroll
      for (int bj = 0; bj < Core::NJ; ++bj)
#pragma unroll
        for (int v = 0; v < 16; ++v)
          if (!EDGE || jw + 32 * bj + 8 * (v >> 2) + (v & 3) < jn) m = fmaxf(m, acc[bj][bi][v]);
      m *= scale;
      // nothing above -inf: every term is exp(-inf) = 0
      const float ms = m == -INFINITY ? 0.0f : m;
      float s = 0.0f;
#pragma unroll
      for (int bj = 0; bj < Core::NJ; ++bj)
#pragma unroll
        for (int v = 0; v < 16; ++v)
          if (!EDGE || jw + 32 * bj + 8 * (v >> 2) + (v & 3) < jn)
            s += exp_of<T>(__builtin_fmaf(acc[bj][bi][v], scale, -ms));
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
template <bool LISTS, typename Core, typename T>
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
  stats_out<LISTS, Core, T>(a, w, acc);
}

// A product with g: the sum over its planes, `plane` elements apart, the low one
// first, or with TURNS (on the grid) a stage of each in turns, which reads the
// other operand from memory once: distillation step of 57 x 151637 x 3008 1058
// us without and 942 with, 2048 x 32000 x 2048 1559 and 1532, 8192 x 32000 x 2048
// 5650 and 5564, 4096 x 163840 x 7168 46.1 ms and 45.0.
template <bool TURNS, typename Core, typename T>
__device__ __forceinline__ void run_planes(LossTile<T>& w, int64_t plane,
                                           f32x16_t (&acc)[Core::NJ][Core::MI]) {
  if constexpr (sizeof(T) != 2) {
    Core::run(w, acc);
  } else if constexpr (TURNS && Core::kGrid) {
    Core::template run<false, 2>(w, acc, plane);
  } else {
    zero_acc(acc);
#pragma unroll 1
    for (int p = 0; p < 2; ++p, w.P += plane) Core::template run<true>(w, acc);
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
  float scale;
};

// dh (+)= g W of the piece; split s takes its share of the piece's rows.
template <bool TURNS, typename Core, typename T, typename TO>
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
  run_planes<TURNS, Core, T>(w, a.n * a.ldg, acc);
  // no gradient for a row without a target, where a weight is not finite too
  const float c = *a.c * a.scale;
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

struct DwArgs {
  const void* g;
  const void* h;  // k_loss_rows' copy
  const float* c;
  void* dw;  // the piece's first row
  int64_t ldg, ldh, vocab;
  int n, dim, len, accumulate, cols;  // cols: of dw, at most dim
  float scale;
};

// How a tile of dw is stored: in rows on the grid, past the caches (kStream) or
// not, or (kOff) quad by quad.
enum Store { kRows, kStream, kOff };
template <bool TURNS, typename Core, Store STORE, typename T, typename TO>
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
  run_planes<TURNS, Core, T>(w, a.n * a.ldg, acc);
  scale_acc(acc, *a.c * a.scale);
  TO* C = static_cast<TO*>(a.dw) + static_cast<int64_t>(w.i0) * a.cols + w.j0;
  const TO* add = a.accumulate ? C : nullptr;
  if constexpr (STORE == kOff)
    write_quads<Core>(acc, C, a.cols, add, a.cols, w.pn, a.cols - w.j0);
  else
    Core::template write<STORE == kStream>(acc, C, a.cols, add, a.cols, w.pn, a.cols - w.j0);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
auto row_tiles(int64_t rows) {
  return [rows](int bm) { return static_cast<double>(ceil_div(rows, bm)); };
}
// dh: `splits` times the tiles, each with its share of the sum
auto dh_tiles(int64_t n, int splits) {
  return [n, splits](int bm) { return static_cast<double>(ceil_div(n, bm) * splits); };
}

// bf16 operands on the 16-byte grid take the DMA core (grid), others the
// core for any operands.
template <bool LISTS, typename Core, typename T>
int launch_stats(const StatsArgs& a, hipStream_t s) {
  const int nx = static_cast<int>(ceil_div(a.n, Core::BM));
  const int ny = static_cast<int>(ceil_div(a.vocab, Core::BN));
  hipLaunchKernelGGL((k_loss_stats<LISTS, Core, T>), dim3(tile_blocks(nx, ny)),
                     dim3(kThreads), 0, s, a, nx, ny);
  return ny;
}
// returns the number of tiles along the vocabulary
template <bool LISTS, typename T>
int run_stats(const StatsArgs& a, bool grid, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (grid) {
      const Shape shape = pick_shape(kShapeNT, row_tiles(a.n), a.vocab, a.dim);
      if (shape == kLarge) return launch_stats<LISTS, LargeCore<false, false>, T>(a, s);
      if (shape == kHalf) return launch_stats<LISTS, HalfCore<false, false>, T>(a, s);
      if (shape == kMedium) return launch_stats<LISTS, MediumCore<false, false>, T>(a, s);
      return launch_stats<LISTS, ThinCore<false, false>, T>(a, s);
    }
  }
  if (pick_any_large<T>(row_tiles(a.n), a.vocab, a.dim))
    return launch_stats<LISTS, OtherCore<T, false, false, 128>, T>(a, s);
  return launch_stats<LISTS, OtherCore<T, false, false, 64>, T>(a, s);
}

template <bool TURNS, typename Core, typename T, typename TO>
void launch_dh(const DhArgs& a, hipStream_t s) {
  const int nx = static_cast<int>(ceil_div(a.n, Core::BM));
  const int ny = static_cast<int>(ceil_div(a.dim, Core::BN));
  hipLaunchKernelGGL((k_loss_dh<TURNS, Core, T, TO>),
                     dim3(tile_blocks(nx, static_cast<int64_t>(ny) * a.splits)),
                     dim3(kThreads), 0, s, a, nx, ny);
}
// bf16: a sum runs over both planes of g
template <typename T>
constexpr int64_t kPlanes = sizeof(T) == 2 ? 2 : 1;
template <bool TURNS, typename T, typename TO>
void run_dh(const DhArgs& a, bool grid, hipStream_t s) {
  const int64_t k = kPlanes<T> * ceil_div(a.len, a.splits);
  if constexpr (sizeof(T) == 2) {
    if (grid) {
      const Shape shape = pick_shape(kShapeNN, dh_tiles(a.n, a.splits), a.dim, k);
      if (shape == kLarge) return launch_dh<TURNS, LargeCore<false, true>, T, TO>(a, s);
      if (shape == kHalf) return launch_dh<TURNS, HalfCore<false, true>, T, TO>(a, s);
      if (shape == kMedium) return launch_dh<TURNS, MediumCore<false, true>, T, TO>(a, s);
      return launch_dh<TURNS, ThinCore<false, true>, T, TO>(a, s);
    }
  }
  if (pick_any_large<T>(dh_tiles(a.n, a.splits), a.dim, k))
    launch_dh<TURNS, OtherCore<T, false, true, 128>, T, TO>(a, s);
  else
    launch_dh<TURNS, OtherCore<T, false, true, 64>, T, TO>(a, s);
}

template <bool TURNS, typename Core, typename T, typename TO>
void launch_dw(const DwArgs& a, hipStream_t s) {
  const int nx = static_cast<int>(ceil_div(a.len, Core::BM));
  const int ny = static_cast<int>(ceil_div(a.dim, Core::BN));
  auto* kernel = k_loss_dw<TURNS, Core, kRows, T, TO>;
  if constexpr (Core::kGrid) {
    if (stream_gradient(static_cast<const TO*>(a.dw), a.vocab, a.cols))
      kernel = k_loss_dw<TURNS, Core, kStream, T, TO>;
    if constexpr (TURNS) {
      if (!on_grid(a.dw, a.cols, a.cols)) kernel = k_loss_dw<TURNS, Core, kOff, T, TO>;
    }
  }
  hipLaunchKernelGGL(kernel, dim3(tile_blocks(nx, ny)), dim3(kThreads), 0, s, a, nx, ny);
}
template <bool TURNS, typename T, typename TO>
void run_dw(const DwArgs& a, bool grid, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (grid) {
      const Shape shape = pick_shape(kShapeTN, row_tiles(a.len), a.dim, kPlanes<T> * a.n);
      if (shape == kLarge) return launch_dw<TURNS, LargeCore<true, true>, T, TO>(a, s);
      if (shape == kHalf) return launch_dw<TURNS, HalfCore<true, true>, T, TO>(a, s);
      return launch_dw<TURNS, MediumCore<true, true>, T, TO>(a, s);
    }
  }
  if (pick_any_large<T>(row_tiles(a.len), a.dim, kPlanes<T> * a.n))
    launch_dw<TURNS, OtherCore<T, true, true, 128>, T, TO>(a, s);
  else
    launch_dw<TURNS, OtherCore<T, true, true, 64>, T, TO>(a, s);
}

template <typename T>
constexpr int32_t kType = sizeof(T) == 2 ? MUON_DTYPE_BF16 : MUON_DTYPE_FP32;
template <bool LISTS, typename T, typename TH, typename TW>
void run_backward(const BackwardArgs& b, const LossWs& w, hipStream_t s) {
  T* g = reinterpret_cast<T*>(b.ws + w.g);
  float* part = reinterpret_cast<float*>(b.ws + w.part);
  float* c = reinterpret_cast<float*>(b.ws + w.c);
  loss_scale(b, c, s);
  T* rows = reinterpret_cast<T*>(b.ws + w.rows);
  if constexpr (!LISTS) {
    if (b.dw != nullptr) loss_rows(b, rows, kType<T>, s);
  }
  const bool grid = on_grid(b.h, b.ldh, b.dim) && on_grid(b.w, b.dim, b.dim);
  // operands laid out on the grid for results that are not: dh leaves the fp32
  // sums in the join alone, dw's tiles are stored quad by quad
  const bool laid = LISTS && b.cols != b.dim;
  for (int64_t v0 = 0; v0 < b.vocab; v0 += w.piece) {
    const int len = static_cast<int>(std::min(w.piece, b.vocab - v0));
    const T* wp = static_cast<const T*>(b.w) + v0 * b.dim;
    loss_g(GradArgs{b.h, wp, b.targets, b.lse, b.dloss, c, g, b.ldh, w.ldg, b.vocab, v0,
                    static_cast<int>(b.n), static_cast<int>(b.dim), len, b.t64, b.scale},
           kType<T>, grid, s);
    if (b.after_g != nullptr) b.after_g(b.context, g, w.ldg, c, v0, len, s);
    if (b.dh != nullptr) {
      const bool last = v0 + len == b.vocab;
      run_dh<LISTS, T, TH>(
          DhArgs{g, wp, b.targets, c, part, last && w.splits == 1 && !laid ? b.dh : nullptr, w.ldg,
                 b.ld_dh, b.vocab, static_cast<int>(b.n), static_cast<int>(b.dim), len, w.splits,
                 v0 == 0 ? 1 : 0, b.t64, b.scale},
          grid && (laid || on_grid(b.dh, b.ld_dh, b.dim)), s);
    }
    if (b.dw != nullptr)
      run_dw<LISTS, T, TW>(
          DwArgs{g, rows, c, static_cast<TW*>(b.dw) + v0 * b.cols, w.ldg, b.dim, b.vocab,
                 static_cast<int>(b.n), static_cast<int>(b.dim), len, b.accumulate,
                 static_cast<int>(b.cols), b.scale},
          grid && (laid || on_grid(b.dw, b.dim, b.dim)), s);
  }
  if (b.dh != nullptr && (w.splits > 1 || laid))
    loss_dh_join(part, w.splits, static_cast<int>(b.n), static_cast<int>(b.dim),
                 static_cast<int>(b.cols), b.dh, kType<TH>, b.ld_dh, s);
}

// Row statistics of scale * h W^T, and what targets or keys name.  Returns the
// number of tiles along the vocabulary.
template <bool LISTS>
int loss_stats(const StatsArgs& a, int32_t dtype, hipStream_t s) {
  const bool grid = on_grid(a.h, a.ldh, a.dim) && on_grid(a.w, a.dim, a.dim);
  return dtype == MUON_DTYPE_BF16 ? run_stats<LISTS, uint16_t>(a, grid, s)
                                  : run_stats<LISTS, float>(a, grid, s);
}

template <bool LISTS>
void loss_backward(const BackwardArgs& b, const LossWs& w, int32_t dtype, int32_t dh_dtype,
                   int32_t dw_dtype, hipStream_t s) {
  const bool hb = dh_dtype == MUON_DTYPE_BF16, wb = dw_dtype == MUON_DTYPE_BF16;
  auto run = [&](auto t) {
    using T = decltype(t);
    if (hb && wb) run_backward<LISTS, T, uint16_t, uint16_t>(b, w, s);
    else if (hb) run_backward<LISTS, T, uint16_t, float>(b, w, s);
    else if (wb) run_backward<LISTS, T, float, uint16_t>(b, w, s);
    else run_backward<LISTS, T, float, float>(b, w, s);
  };
  if (dtype == MUON_DTYPE_BF16) run(uint16_t{});
  else run(float{});
}

}  // namespace
}  // namespace muon
