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

#include "lm_loss_kernels.h"

namespace muon {
namespace {

template <int R>
__global__ __launch_bounds__(kThreads) void k_loss_join(const float* __restrict__ tile_m,
                                                        const float* __restrict__ tile_s,
                                                        const float* __restrict__ at, int tiles,
                                                        int n, const void* targets, int t64,
                                                        int64_t vocab, float* __restrict__ loss,
                                                        float* __restrict__ lse) {
  const int t = blockIdx.x * R + threadIdx.x % R;
  float m, s;
  join_tiles<R>(tile_m, tile_s, tiles, n, t, m, s);
  if (threadIdx.x >= R || t >= n) return;
  // (m - at) + log s, not lse - at: the rounding of lse, half a step of m, is
  // all there is of a likely target's loss
  const float ls = logf(s);
  lse[t] = m + ls;
  loss[t] = target_of(targets, t64, t, vocab) >= 0 ? (m - at[t]) + ls : 0.0f;
}

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
        const float p = exp_of<T>(__builtin_fmaf(acc[bj][bi][v], a.scale, -lse[bi]));
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

template <typename TO>
__global__ __launch_bounds__(kThreads) void k_loss_dh_join(const float* __restrict__ part,
                                                           int splits, int n, int dim, int cols,
                                                           TO* out, int64_t ld) {
  const int64_t total = static_cast<int64_t>(n) * dim;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    float v = part[i];
#pragma unroll 8
    for (int s = 1; s < splits; ++s) v += part[s * total + i];
    const int64_t t = i / dim;
    const int d = static_cast<int>(i - t * dim);
    if (d < cols) from_f32(v, out + t * ld + d);
  }
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

}  // namespace

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

int loss_no_rows(void* dw, int32_t dw_dtype, int64_t vocab, int64_t dim, int accumulate,
                 hipStream_t s) {
  if (dw == nullptr || accumulate) return MUON_OK;
  if (dw_dtype == MUON_DTYPE_BF16)
    hipLaunchKernelGGL(k_zero_rows<uint16_t>, dim3(4096), dim3(kThreads), 0, s,
                       static_cast<uint16_t*>(dw), vocab, dim, dim);
  else
    hipLaunchKernelGGL(k_zero_rows<float>, dim3(4096), dim3(kThreads), 0, s,
                       static_cast<float*>(dw), vocab, dim, dim);
  return check_launch("vocabulary loss gradient launch");
}

void loss_scale(const BackwardArgs& b, float* c, hipStream_t s) {
  hipLaunchKernelGGL(k_loss_scale, dim3(1), dim3(kScaleThreads), 0, s, b.dloss,
                     static_cast<int>(b.n), b.targets, b.t64, b.vocab, c);
}

void loss_rows(const BackwardArgs& b, void* rows, int32_t dtype, hipStream_t s) {
  auto run = [&](auto t) {
    using T = decltype(t);
    const int64_t pieces = b.n * ceil_div(b.dim, 16 / static_cast<int64_t>(sizeof(T)));
    hipLaunchKernelGGL(k_loss_rows<T>,
                       dim3(static_cast<unsigned>(std::min<int64_t>(8192, ceil_div(pieces, kThreads)))),
                       dim3(kThreads), 0, s, static_cast<const T*>(b.h), b.ldh, b.targets, b.t64,
                       static_cast<int>(b.n), static_cast<int>(b.dim), b.vocab,
                       static_cast<T*>(rows));
  };
  if (dtype == MUON_DTYPE_BF16) run(uint16_t{});
  else run(float{});
}

void loss_g(const GradArgs& a, int32_t dtype, bool grid, hipStream_t s) {
  if (dtype == MUON_DTYPE_BF16) run_g<uint16_t>(a, grid, s);
  else run_g<float>(a, grid, s);
}

void loss_dh_join(const float* part, int splits, int n, int dim, int cols, void* out,
                  int32_t out_dtype, int64_t ld, hipStream_t s) {
  const int64_t total = static_cast<int64_t>(n) * dim;
  const dim3 blocks(static_cast<unsigned>(std::min<int64_t>(4096, ceil_div(total, kThreads))));
  if (out_dtype == MUON_DTYPE_BF16)
    hipLaunchKernelGGL(k_loss_dh_join<uint16_t>, blocks, dim3(kThreads), 0, s, part, splits, n, dim,
                       cols, static_cast<uint16_t*>(out), ld);
  else
    hipLaunchKernelGGL(k_loss_dh_join<float>, blocks, dim3(kThreads), 0, s, part, splits, n, dim,
                       cols, static_cast<float*>(out), ld);
}

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
    StatsArgs a{};
    a.h = static_cast<const char*>(hidden) + static_cast<size_t>(r0 * ld_hidden) * sz;
    a.w = weight;
    a.targets = tg;
    a.tile_m = tm;
    a.tile_s = ts;
    a.at = at;
    a.ldh = ld_hidden;
    a.vocab = vocab;
    a.n = rows;
    a.dim = static_cast<int>(dim);
    a.t64 = targets_64 != 0;
    a.scale = 1.0f;
    const int v_tiles = loss_stats<false>(a, dtype, stream);
    const int per = join_rows(rows);
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
  // no rows: dweight is a sum of nothing
  if (n == 0) return loss_no_rows(dweight, dweight_dtype, vocab, dim, accumulate, stream);
  if (dhidden == nullptr && dweight == nullptr) return MUON_OK;
  if (hidden == nullptr || weight == nullptr || targets == nullptr || lse == nullptr ||
      dloss == nullptr)
    return set_error(MUON_ERR_INVALID_ARG, "hidden, weight, targets, lse or dloss is null");
  const LossWs w = loss_ws(n, vocab, dim, dtype, true);
  if ((rc = check_ws(workspace, workspace_bytes, w.total, "lm_loss_backward")) != MUON_OK) return rc;
  BackwardArgs b{};
  b.h = hidden;
  b.w = weight;
  b.targets = targets;
  b.lse = lse;
  b.dloss = dloss;
  b.dh = dhidden;
  b.dw = dweight;
  b.n = n;
  b.vocab = vocab;
  b.dim = dim;
  b.ldh = ld_hidden;
  b.ld_dh = ld_dhidden;
  b.cols = dim;
  b.t64 = targets_64 != 0;
  b.accumulate = accumulate != 0;
  b.ws = static_cast<char*>(workspace);
  b.scale = 1.0f;
  loss_backward<false>(b, w, dtype, dhidden_dtype, dweight_dtype, stream);
  return check_launch("vocabulary loss gradient launch");
}

}  // extern "C"
