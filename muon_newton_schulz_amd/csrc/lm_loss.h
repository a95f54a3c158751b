// What losses of a linear head over a large vocabulary share, the cross
// entropy (lm_loss.hip, which defines the functions) and the distillation loss
// (distill.hip), besides their kernels (lm_loss_kernels.h).
#pragma once

#include "train_common.h"

namespace muon {

// (m, s) <- (m, s) + (m2, s2): sums of exp(l - m) over disjoint sets.  A set
// without a value above -inf has s = 0.
__device__ __forceinline__ void join_stats(float& m, float& s, float m2, float s2) {
  const float mm = fmaxf(m, m2);
  const float a = m == mm ? s : s * expf(m - mm);
  const float b = m2 == mm ? s2 : s2 * expf(m2 - mm);
  m = mm;
  s = a + b;
}

// Joins the tile statistics of row t (below n) in a fixed order: thread (r, p)
// of a workgroup of 256 takes tiles p, p + P, ... of row r, R rows x P parts,
// then the parts are joined pairwise.  Rows run along the lanes, so loads of
// many rows are whole lines; few rows take more parts.  The result is that of
// the threads of part 0.
template <int R>
__device__ __forceinline__ void join_tiles(const float* __restrict__ tile_m,
                                           const float* __restrict__ tile_s, int tiles, int n,
                                           int t, float& m, float& s) {
  constexpr int P = 256 / R;
  __shared__ float red[4][R][2];
  const int r = threadIdx.x % R, part = threadIdx.x / R;
  m = -INFINITY;
  s = 0.0f;
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
  for (int p = 1; p < 4; ++p) join_stats(m, s, red[p][r][0], red[p][r][1]);
}
// Rows to a workgroup: 16, or 4 (and 64 parts) where there are few rows (the
// cross entropy's call: 33 x 32000 x 2048 27.1 us against 29.7, 512 x 163840 x
// 64 40.1 against 40.5, but 2048 x 32000 x 64 34.6 against 30.8).
inline int join_rows(int rows) { return rows <= 512 ? 4 : 16; }

// ---- host side (lm_loss.hip) ----

// Workspace layout: of a forward, or with backward of both.
struct LossWs {
  int64_t stats_rows, v_tiles;          // forward
  int64_t piece, ldg;                   // backward
  int splits;
  size_t tile_m, tile_s, at, c, g, rows, part, total;
};
LossWs loss_ws(int64_t n, int64_t vocab, int64_t dim, int32_t dtype, bool backward);

int check_loss(int64_t n, int64_t vocab, int64_t dim, int64_t ldh, int32_t dtype);
int check_ws(const void* ws, size_t bytes, size_t need, const char* who);

// A row's listed columns: their keys (column << 10 | place in the list, at
// most 2^10 places of 2^21 columns), ascending, and ~0 where the list ends.
constexpr int kPlaceBits = 10;
struct StatsArgs {
  const void* h;
  const void* w;
  const void* targets;   // or null
  float* tile_m;         // [vocabulary tiles][n], of scale * logits
  float* tile_s;
  float* at;             // [n], the target's logit
  const uint32_t* keys;  // [n][top], or null
  float* points;         // [n][top], the listed columns' logits, not scaled
  int64_t ldh, vocab;
  int n, dim, t64, top;
  float scale;           // of the logits, > 0
};

// Gradients with g = (exp(scale l - lse) - [v = target]) dloss scale.  after_g
// is called when a piece's g / (scale c) is stored ([n][ldg], columns
// [v0, v0 + len); bf16: a low plane, then a high plane), to put other values
// into it.  The distillation loss has put hidden, with zeros in the rows
// without a target, into the workspace already.
struct BackwardArgs {
  const void *h, *w, *targets;
  const float *lse, *dloss;
  void *dh, *dw;  // either may be null
  int64_t n, vocab, dim, ldh, ld_dh;
  int64_t cols;   // of dh and dw, at most dim: operands may be laid out with more
  int t64, accumulate;
  char* ws;
  float scale;
  void (*after_g)(const void* context, void* g, int64_t ldg, const float* c, int64_t v0, int len,
                  hipStream_t s);
  const void* context;
};
// c: the largest finite |dloss| of the rows with a target, 1 if that is 0.
void loss_scale(const BackwardArgs& b, float* c, hipStream_t s);
// hidden with zeros in the rows without a target, [n][dim]: dW's sum runs over
// all rows, and 0 times what such a row holds is 0 only where that is finite.
void loss_rows(const BackwardArgs& b, void* rows, int32_t dtype, hipStream_t s);
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
  float scale;           // of the logits
};
// g / c of a piece; grid: the operands are on the DMA core's grid
void loss_g(const GradArgs& a, int32_t dtype, bool grid, hipStream_t s);
// dhidden = sum of the splits [splits][n][dim], in order; of the sums' dim columns
// the first cols.
void loss_dh_join(const float* part, int splits, int n, int dim, int cols, void* out,
                  int32_t out_dtype, int64_t ld, hipStream_t s);
// dw (+)= nothing, for calls without rows
int loss_no_rows(void* dw, int32_t dw_dtype, int64_t vocab, int64_t dim, int accumulate,
                 hipStream_t s);

}  // namespace muon
