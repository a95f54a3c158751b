// Matrix products grouped by expert, with ragged group sizes.
//
//   y_r  = x_r W_e   or  x_r W_e^T       for offsets[e] <= r < offsets[e+1]
//   dW_e = sum over those r of a_r^T b_r                     (+ dW_e)
//
// The group sizes are device data: no call reads them on the host.  Every
// workgroup of a product finds its expert and row tile by a scan of the
// offsets; the launch has as many row tiles as any sizes can need.
#include <algorithm>

#include "train_gemm.h"

namespace muon {
namespace {

constexpr int kThreads = 256;

// Rows of expert e, whatever the offsets hold: within [0, rows), never
// negative.
__device__ __forceinline__ void group_rows(const int32_t* off, int e, int rows, int& lo, int& n) {
  lo = min(max(off[e], 0), rows);
  n = max(min(off[e + 1], rows) - lo, 0);
}

struct RowTile {
  int e, lo, n, tile;  // expert, its first row and row count, tile within it
};
// Row tiles of all groups, each cut into tiles of bm rows; with find also the
// t-th of them.  Every wave scans the offsets, 64 experts at a time.
template <bool FIND>
__device__ __forceinline__ int scan_row_tiles(const int32_t* off, int experts, int rows, int bm,
                                              int t, RowTile* out) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int e0 = 0; e0 < experts; e0 += 64) {
    int lo = 0, n = 0;
    if (e0 + lane < experts) group_rows(off, e0 + lane, rows, lo, n);
    const int tiles = (n + bm - 1) / bm;
    int s = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(s, o, 64);
      if (lane >= o) s += u;
    }
    if constexpr (FIND) {
      const uint64_t over = __ballot(base + s > t);
      if (over != 0) {
        // uniform values, in scalar registers
        const int l = __ffsll(static_cast<unsigned long long>(over)) - 1;
        out->e = e0 + l;
        out->lo = __builtin_amdgcn_readlane(lo, l);
        out->n = __builtin_amdgcn_readlane(n, l);
        out->tile = t - base - __builtin_amdgcn_readlane(s - tiles, l);
        return 0;
      }
    }
    base += __builtin_amdgcn_readlane(s, 63);
  }
  return base;
}

// Row tiles that any group sizes can need.
__host__ __device__ __forceinline__ int most_row_tiles(int rows, int experts, int bm) {
  return rows / bm + (experts < rows ? experts : rows);
}

struct MatmulArgs {
  const void* x;
  const void* w;
  void* y;
  const int32_t* off;
  int64_t ldx, ldy;
  int experts, rows, K, N;
};

// QKS: W_e is [K][N] (y = x W_e); else [N][K] (y = x W_e^T).  The launch has
// as many workgroups as any sizes can need; they share the tiles that the
// offsets give.
template <typename T>
struct MatmulTile : TileArgs<T> {
  int64_t row0;
  int j0;
};
template <typename Core, typename T, bool QKS, typename TO>
__global__ __launch_bounds__(kThreads, Core::kWaves) void k_expert_matmul(MatmulArgs a, int ny) {
  using W = MatmulTile<T>;
  // (offsets out of order can give any number of tiles: no more than the
  // launch's are taken)
  const int nx = min(scan_row_tiles<false>(a.off, a.experts, a.rows, Core::BM, 0, nullptr),
                     most_row_tiles(a.rows, a.experts, Core::BM));
  int x, y;
  if (!my_tile(nx, ny, x, y)) return;
  W w;
  RowTile rt;
  scan_row_tiles<true>(a.off, a.experts, a.rows, Core::BM, x, &rt);
  const int i0 = rt.tile * Core::BM;
  w.j0 = y * Core::BN;
  w.row0 = static_cast<int64_t>(rt.lo) + i0;
  w.P = static_cast<const T*>(a.x) + w.row0 * a.ldx;
  w.ldp = a.ldx;
  w.pn = rt.n - i0;
  w.Q = static_cast<const T*>(a.w) + static_cast<int64_t>(rt.e) * a.K * a.N +
        (QKS ? w.j0 : static_cast<int64_t>(w.j0) * a.K);
  w.ldq = QKS ? a.N : a.K;
  w.qn = a.N - w.j0;
  w.K = a.K;
  f32x16_t acc[Core::NJ][Core::MI];
  Core::run(w, acc);
  Core::write(acc, static_cast<TO*>(a.y) + w.row0 * a.ldy + w.j0, a.ldy,
              static_cast<const TO*>(nullptr), 0, w.pn, w.qn);
}

struct WgradArgs {
  const void* a;
  const void* b;
  void* dw;
  const int32_t* off;
  int64_t lda, ldb;
  int experts, rows, M, N, accumulate;
};

// Zeros for a tile on the 16-byte grid (64 experts, 8 rows, 2048 x 1408: with
// the streamed stores of a tile of zeros 69 us, so 59).
template <typename Core, typename TO>
__device__ __forceinline__ void zero_tile(TO* C, int64_t ldc, int rows, int cols) {
  constexpr int E = 16 / sizeof(TO), CPR = Core::BN / E;
#pragma unroll 4
  for (int k = threadIdx.x; k < Core::BM * CPR; k += kThreads) {
    const int i = k / CPR, j = k % CPR * E;
    if (i < rows && j < cols) *reinterpret_cast<u32x4_t*>(C + i * ldc + j) = u32x4_t{0, 0, 0, 0};
  }
}

template <typename T>
struct WgradTile : TileArgs<T> {
  int64_t out;
};
template <typename Core, bool STREAM, typename T, typename TO>
__global__ __launch_bounds__(kThreads, Core::kWaves) void k_expert_wgrad(WgradArgs g, int nx,
                                                                       int ny) {
  using W = WgradTile<T>;
  int x, y;
  if (!my_tile(static_cast<int64_t>(nx) * g.experts, ny, x, y)) return;
  W w;
  const int e = x / nx, i0 = x % nx * Core::BM, j0 = y * Core::BN;
  int lo, n;
  group_rows(g.off, e, g.rows, lo, n);
  if (n == 0 && g.accumulate) return;
  if constexpr (Core::kGrid) {
    if (n == 0) {
      zero_tile<Core>(static_cast<TO*>(g.dw) + (static_cast<int64_t>(e) * g.M + i0) * g.N + j0,
                      g.N, g.M - i0, g.N - j0);
      return;
    }
  }
  w.P = static_cast<const T*>(g.a) + lo * g.lda + i0;
  w.ldp = g.lda;
  w.pn = g.M - i0;
  w.Q = static_cast<const T*>(g.b) + lo * g.ldb + j0;
  w.ldq = g.ldb;
  w.qn = g.N - j0;
  w.K = n;
  w.out = (static_cast<int64_t>(e) * g.M + i0) * g.N + j0;
  f32x16_t acc[Core::NJ][Core::MI];
  Core::run(w, acc);
  TO* C = static_cast<TO*>(g.dw) + w.out;
  Core::template write<STREAM>(acc, C, g.N, g.accumulate ? C : static_cast<const TO*>(nullptr), g.N,
                               w.pn, w.qn);
}

// -------------------------------------------------------------------- host

constexpr int kMaxExperts = 4096;

// Narrow matrices of many experts with a side of millions can need more tiles
// than a launch holds.
int refuse_tiles() {
  return set_error(MUON_ERR_UNSUPPORTED, "more result tiles than a launch holds (2^24)");
}
template <typename Core, typename T, bool QKS, typename TO>
int launch_matmul(const MatmulArgs& a, hipStream_t s) {
  const int nx = most_row_tiles(a.rows, a.experts, Core::BM);
  const int ny = (a.N + Core::BN - 1) / Core::BN;
  if (!tiles_fit(nx, ny)) return refuse_tiles();
  hipLaunchKernelGGL((k_expert_matmul<Core, T, QKS, TO>),
                     dim3(tile_blocks(nx, ny)), dim3(kThreads), 0, s, a, ny);
  return check_launch("expert product launch");
}
template <typename Core, typename T, typename TO>
int launch_wgrad(const WgradArgs& g, hipStream_t s) {
  const int nx = (g.M + Core::BM - 1) / Core::BM, ny = (g.N + Core::BN - 1) / Core::BN;
  if (!tiles_fit(static_cast<int64_t>(nx) * g.experts, ny)) return refuse_tiles();
  auto* kernel = k_expert_wgrad<Core, false, T, TO>;
  if constexpr (Core::kGrid) {
    if (stream_gradient(static_cast<const TO*>(g.dw), static_cast<int64_t>(g.experts) * g.M, g.N))
      kernel = k_expert_wgrad<Core, true, T, TO>;
  }
  hipLaunchKernelGGL(kernel, dim3(tile_blocks(static_cast<int64_t>(nx) * g.experts, ny)),
                     dim3(kThreads), 0, s, g, nx, ny);
  return check_launch("expert weight gradient launch");
}

// Row tiles of the groups, whose sizes the host does not know: rows spread
// evenly, and half a tile lost at each group's end.
double group_tiles(int rows, int experts, int bm) {
  const double groups = std::min(rows, experts), r = rows / groups;
  return groups * (r <= bm / 2 ? 1.0 : r / bm + 0.6);
}

template <bool QKS, typename TO>
int run_matmul_grid(const MatmulArgs& a, hipStream_t s) {
  const Shape shape = pick_shape(QKS ? kShapeNN : kShapeNT, [&](int bm) {
    return group_tiles(a.rows, a.experts, bm);
  }, a.N, a.K);
  using T = uint16_t;
  if (shape == kLarge) return launch_matmul<LargeCore<false, QKS>, T, QKS, TO>(a, s);
  if (shape == kHalf) return launch_matmul<HalfCore<false, QKS>, T, QKS, TO>(a, s);
  if (shape == kMedium) return launch_matmul<MediumCore<false, QKS>, T, QKS, TO>(a, s);
  return launch_matmul<ThinCore<false, QKS>, T, QKS, TO>(a, s);
}

template <typename T, typename TO>
int run_matmul(const MatmulArgs& a, bool trans, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (on_grid(a.x, a.ldx, a.K) && on_grid(a.w, a.N, a.K) && on_grid(a.y, a.ldy, a.N)) {
      return trans ? run_matmul_grid<false, TO>(a, s) : run_matmul_grid<true, TO>(a, s);
    }
  }
  const bool large = pick_any_large<T>(
      [&](int bm) { return group_tiles(a.rows, a.experts, bm); }, a.N, a.K);
  if (trans) {
    if (large) return launch_matmul<OtherCore<T, false, false, 128>, T, false, TO>(a, s);
    return launch_matmul<OtherCore<T, false, false, 64>, T, false, TO>(a, s);
  }
  if (large) return launch_matmul<OtherCore<T, false, true, 128>, T, true, TO>(a, s);
  return launch_matmul<OtherCore<T, false, true, 64>, T, true, TO>(a, s);
}

template <typename T, typename TO>
int run_wgrad(const WgradArgs& g, hipStream_t s) {
  auto tiles = [&](int bm) { return static_cast<double>(g.experts) * ((g.M + bm - 1) / bm); };
  const int64_t k = g.rows / g.experts;
  if constexpr (sizeof(T) == 2) {
    if (on_grid(g.a, g.lda, g.M) && on_grid(g.b, g.ldb, g.N) && on_grid(g.dw, g.N, g.M)) {
      const Shape shape = pick_shape(kShapeTN, tiles, g.N, k);
      if (shape == kLarge) return launch_wgrad<LargeCore<true, true>, T, TO>(g, s);
      if (shape == kHalf) return launch_wgrad<HalfCore<true, true>, T, TO>(g, s);
      return launch_wgrad<MediumCore<true, true>, T, TO>(g, s);
    }
  }
  if (pick_any_large<T>(tiles, g.N, k))
    return launch_wgrad<OtherCore<T, true, true, 128>, T, TO>(g, s);
  return launch_wgrad<OtherCore<T, true, true, 64>, T, TO>(g, s);
}

int check_group(int64_t rows, int32_t experts, int64_t k, int64_t n) {
  if (rows < 0 || rows > kMaxTokens)
    return set_error(MUON_ERR_BAD_SHAPE, "rows must be in [0, 2^26)");
  if (experts < 1 || experts > kMaxExperts)
    return set_error(MUON_ERR_BAD_SHAPE, "experts must be in [1, 4096]");
  if (k < 1 || k > (1 << 22) || n < 1 || n > (1 << 22))
    return set_error(MUON_ERR_BAD_SHAPE, "a weight's sides must be in [1, 2^22]");
  return MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

int expert_matmul(const void* x, int64_t ldx, const void* w, int32_t dtype,
                  const int32_t* offsets, int32_t experts, int64_t rows, int64_t k, int64_t n,
                  int32_t trans_w, void* y, int32_t y_dtype, int64_t ldy, hipStream_t stream) {
  const int rc = check_group(rows, experts, k, n);
  if (rc != MUON_OK) return rc;
  if (!train_dtype_ok(dtype) || !train_dtype_ok(y_dtype))
    return set_error(MUON_ERR_BAD_DTYPE, "x, w and y must be fp32 or bf16");
  if (ldx < k || ldy < n) return set_error(MUON_ERR_BAD_SHAPE, "ldx < k or ldy < n");
  if (rows == 0) return MUON_OK;
  if (x == nullptr || w == nullptr || offsets == nullptr || y == nullptr)
    return set_error(MUON_ERR_INVALID_ARG, "x, w, offsets or y is null");
  const MatmulArgs a{x, w, y, offsets, ldx, ldy, experts, static_cast<int>(rows),
                     static_cast<int>(k), static_cast<int>(n)};
  const bool tr = trans_w != 0, yb = y_dtype == MUON_DTYPE_BF16;
  if (dtype == MUON_DTYPE_BF16)
    return yb ? run_matmul<uint16_t, uint16_t>(a, tr, stream)
              : run_matmul<uint16_t, float>(a, tr, stream);
  return yb ? run_matmul<float, uint16_t>(a, tr, stream) : run_matmul<float, float>(a, tr, stream);
}

int expert_wgrad(const void* a, int64_t lda, const void* b, int64_t ldb, int32_t dtype,
                 const int32_t* offsets, int32_t experts, int64_t rows, int64_t m, int64_t n,
                 void* dw, int32_t dw_dtype, int32_t accumulate, hipStream_t stream) {
  const int rc = check_group(rows, experts, m, n);
  if (rc != MUON_OK) return rc;
  if (!train_dtype_ok(dtype) || !train_dtype_ok(dw_dtype))
    return set_error(MUON_ERR_BAD_DTYPE, "a, b and dw must be fp32 or bf16");
  if (lda < m || ldb < n) return set_error(MUON_ERR_BAD_SHAPE, "lda < m or ldb < n");
  if (dw == nullptr || offsets == nullptr)
    return set_error(MUON_ERR_INVALID_ARG, "dw or offsets is null");
  if (rows > 0 && (a == nullptr || b == nullptr))
    return set_error(MUON_ERR_INVALID_ARG, "a or b is null");
  if (rows == 0 && accumulate) return MUON_OK;
  const WgradArgs g{a, b, dw, offsets, lda, ldb, experts, static_cast<int>(rows),
                    static_cast<int>(m), static_cast<int>(n), accumulate != 0};
  const bool wb = dw_dtype == MUON_DTYPE_BF16;
  if (dtype == MUON_DTYPE_BF16)
    return wb ? run_wgrad<uint16_t, uint16_t>(g, stream) : run_wgrad<uint16_t, float>(g, stream);
  return wb ? run_wgrad<float, uint16_t>(g, stream) : run_wgrad<float, float>(g, stream);
}

}  // extern "C"
