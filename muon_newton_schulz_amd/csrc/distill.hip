// Distillation through a linear head: the divergence of the student's softmax
// from a teacher's, which is known at a list of columns a row, without keeping
// the student's logits.
//
//   l_tv    = scale h_t . W_v,  scale = 1 / temperature
//   lse_t   = log sum_v exp l_tv,  logp_tk = l_{t, id_tk} - lse_t
//   q_tk    = exp(scale z_tk) / sum_j exp(scale z_tj)      entries that count
//   loss_t  = sum_k q_tk (log q_tk - logp_tk)
//   g_tv    = (exp(l_tv - lse_t) - sum_{k: id_tk = v} q_tk) dloss_t
//   dh = scale g W,   dW = scale g^T h
//
// An entry counts if its id is a column and its z is above -inf.  A row where
// none does has no loss and no gradient.
//
// The products are the cross entropy's (lm_loss.hip); a list touches few
// of a row's columns, so it is kept out of their inner loops:
//   1. k_distill_sort orders each row's list by column, so that a tile finds
//      its part of it with a search.
//   2. Forward: the statistics' tiles leave the listed columns' logits too, from
//      their registers, so nothing reads W twice.  k_distill_join turns them
//      into log-probabilities beside the join of the row's statistics.
//   3. Backward: the cross entropy's g = exp(l - lse) dloss, and
//      k_distill_points stores what the listed columns have instead, whose
//      exp(logp) the forward left: no logit is computed twice for it, and a
//      column that is listed twice is stored once, with the sum of its q.
#include <algorithm>
#include <cmath>

#include "lm_loss_kernels.h"

namespace muon {
namespace {

constexpr uint32_t kNoKey = ~0u;
constexpr int kMaxTop = 1 << kPlaceBits;
constexpr int kMostSplits = 64;

// The teacher's lists, [n][top] with row strides.
struct Lists {
  const void* ids;
  const void* z;
  int64_t ld_ids, ld_z, vocab;
  int ids64, z16, top;
  float scale;
  // the entry's key, kNoKey if it does not count; its z
  __device__ __forceinline__ uint32_t entry(int64_t t, int k, float& zk) const {
    const int64_t i = t * ld_ids + k;
    const int64_t id = ids64 ? static_cast<const int64_t*>(ids)[i]
                             : static_cast<int64_t>(static_cast<const int32_t*>(ids)[i]);
    zk = value(t, k);
    if (id < 0 || id >= vocab || zk == -INFINITY) return kNoKey;
    return static_cast<uint32_t>(id) << kPlaceBits | static_cast<uint32_t>(k);
  }
  __device__ __forceinline__ float value(int64_t t, int k) const {
    const int64_t j = t * ld_z + k;
    return z16 ? to_f32(static_cast<const uint16_t*>(z)[j]) : static_cast<const float*>(z)[j];
  }
};

// Largest z and log of the sum of exp(scale (z - largest)) over a row's
// entries that count; z: lane's E values, -inf where one does not.
template <int E>
__device__ __forceinline__ void teacher_stats(const float (&z)[E], float scale, float& top,
                                              float& log_sum) {
  bool nan = false;
  top = -INFINITY;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    top = fmaxf(top, z[e]);
    nan |= z[e] != z[e];
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  if (__ballot(nan) != 0) top = NAN;
  float s = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) s += z[e] == -INFINITY ? 0.0f : expf((z[e] - top) * scale);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  log_sum = logf(s);
}

// What the sort leaves besides: (column not null) of row t the first listed
// column or -1, the largest z and log sum; (rows not null) hidden, with column
// zeros for a row without a list, in rows of `room` bytes, zeros behind its own.
struct Marks {
  int32_t* column;
  f32x2_t* stats;
  const char* hidden;
  char* rows;
  int64_t stride, bytes, room;  // of a row
};
// One wave copies a row of `bytes` bytes, elements of two or four, into one of
// `room`; not `some`: zeros.
__device__ __forceinline__ void lay_row(const char* from, char* to, int64_t bytes, int64_t room,
                                        bool some, int lane) {
  for (int64_t i = lane * 16; i < room; i += 64 * 16) {
    if (i + 16 <= bytes) {
      u32x4_t v = {0, 0, 0, 0};
      if (some) __builtin_memcpy(&v, from + i, 16);
      __builtin_memcpy(to + i, &v, 16);
    } else {
      for (int64_t k = i; k < min(i + 16, room); k += 2) {
        uint16_t v = 0;
        if (some && k < bytes) __builtin_memcpy(&v, from + k, 2);
        __builtin_memcpy(to + k, &v, 2);
      }
    }
  }
}

// One wave a row: keys [n][top] in ascending order (a bitonic network over
// 64 E keys, element lane E + e in register e), and what marks asks for.
template <int E>
__global__ __launch_bounds__(kThreads) void k_distill_sort(Lists a, int64_t n, uint32_t* keys,
                                                           Marks marks) {
  const int lane = threadIdx.x & 63;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6);
  if (t >= n) return;
  uint32_t x[E];
  float z[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int k = 64 * e + lane;  // any order will do
    x[e] = kNoKey;
    z[e] = -INFINITY;
    if (k < a.top) {
      float zk;
      x[e] = a.entry(t, k, zk);
      if (x[e] != kNoKey) z[e] = zk;
    }
  }
  if (marks.column != nullptr) {
    float top, log_sum;
    teacher_stats<E>(z, a.scale, top, log_sum);
    if (lane == 0) marks.stats[t] = f32x2_t{top, log_sum};
  }
#pragma unroll
  for (int k = 2; k <= 64 * E; k <<= 1) {
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      if (j >= E) {
        const bool low = ((lane * E) & j) == 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t y = __shfl_xor(x[e], j / E, 64);
          const bool up = ((lane * E + e) & k) == 0;
          x[e] = low == up ? min(x[e], y) : max(x[e], y);
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if ((e & j) != 0) continue;
          const bool up = ((lane * E + e) & k) == 0;
          const uint32_t lo = min(x[e], x[e | j]), hi = max(x[e], x[e | j]);
          x[e] = up ? lo : hi;
          x[e | j] = up ? hi : lo;
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = lane * E + e;
    if (i < a.top) keys[t * a.top + i] = x[e];
  }
  const bool listed =
      marks.column == nullptr || __builtin_amdgcn_readfirstlane(x[0]) != kNoKey;
  if (marks.column != nullptr && lane == 0)
    marks.column[t] = listed ? static_cast<int32_t>(x[0] >> kPlaceBits) : -1;
  if (marks.rows != nullptr)
    lay_row(marks.hidden + t * marks.stride, marks.rows + t * marks.room, marks.bytes, marks.room,
            listed, lane);
}

// The weight's rows laid out in rows of `room` bytes, a wave a row.
__global__ __launch_bounds__(kThreads) void k_distill_lay(const char* w, int64_t rows,
                                                          int64_t bytes, int64_t room, char* out) {
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6);
       r < rows; r += static_cast<int64_t>(gridDim.x) * (kThreads / 64))
    lay_row(w + r * bytes, out + r * room, bytes, room, true, threadIdx.x & 63);
}

// Joins a row's tiles (R rows a workgroup) and turns its listed logits into
// log-probabilities; a wave takes R / 4 rows.
// logp = (scale l - m) - log s, not scale l - lse, and the loss from log q -
// logp: the rounding of lse, half a step of m, would be most of the loss of a
// student that is near its teacher.
template <int R, int E>
__global__ __launch_bounds__(kThreads) void k_distill_join(const float* __restrict__ tile_m,
                                                           const float* __restrict__ tile_s,
                                                           int tiles, int n, Lists a, float* loss,
                                                           float* lse, float* logp) {
  __shared__ float row[R][2];
  const int t0 = blockIdx.x * R;
  {
    const int t = t0 + threadIdx.x % R;
    float m, s;
    join_tiles<R>(tile_m, tile_s, tiles, n, t, m, s);
    if (threadIdx.x < R && t < n) {
      const float ls = logf(s);
      row[threadIdx.x][0] = m;
      row[threadIdx.x][1] = ls;
      lse[t] = m + ls;
    }
  }
  __syncthreads();
  const int lane = threadIdx.x & 63;
  for (int r = threadIdx.x >> 6; r < R; r += kThreads / 64) {
    const int64_t t = t0 + r;
    if (t >= n) break;
    float z[E], l[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int k = 64 * e + lane;
      z[e] = -INFINITY;
      l[e] = 0.0f;
      if (k < a.top) {
        float zk;
        if (a.entry(t, k, zk) != kNoKey) {
          z[e] = zk;
          l[e] = logp[t * a.top + k];
        }
      }
    }
    const float m = row[r][0], ls = row[r][1];
    float top, log_sum, sum = 0.0f;
    teacher_stats<E>(z, a.scale, top, log_sum);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int k = 64 * e + lane;
      if (k >= a.top) continue;
      const bool counts = !(z[e] == -INFINITY);
      const float lp = counts ? __builtin_fmaf(l[e], a.scale, -m) - ls : 0.0f;
      logp[t * a.top + k] = lp;
      const float lq = (z[e] - top) * a.scale - log_sum, q = expf(lq);
      if (counts && !(q == 0.0f)) sum += q * (lq - lp);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
    if (lane == 0) loss[t] = sum;
  }
}

struct PointArgs {
  Lists lists;
  const uint32_t* keys;
  const f32x2_t* stats;
  const float* logp;
  const float* dloss;
  int64_t n;
  int fp32;
};

// The listed columns of a piece of g: (exp(logp) - sum of q) dloss / c, as
// g is held (bf16: low and high plane).  A thread an entry; the first of a
// column's entries stores.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_distill_points(PointArgs a, T* g, int64_t ldg,
                                                             const float* c, int64_t v0, int len) {
  const int top = a.lists.top;
  const int64_t total = a.n * top;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const uint32_t key = a.keys[i];
    const int64_t v = key >> kPlaceBits;
    if (key == kNoKey || v < v0 || v >= v0 + len) continue;
    const int64_t t = i / top;
    const int p = static_cast<int>(i - t * top);
    if (p > 0 && a.keys[i - 1] >> kPlaceBits == v) continue;
    const f32x2_t st = a.stats[t];
    float q = 0.0f;
    for (int64_t j = i; j < i - p + top; ++j) {
      const uint32_t kj = a.keys[j];
      if (kj >> kPlaceBits != v) break;
      const float z = a.lists.value(t, kj & (kMaxTop - 1));
      q += expf((z - st[0]) * a.lists.scale - st[1]);
    }
    const float lp = a.logp[t * top + (key & (kMaxTop - 1))];
    const float x = (expf(lp) - q) * (a.dloss[t] / *c);
    T* at = g + t * ldg + (v - v0);
    if constexpr (sizeof(T) == 2) {
      const uint16_t hi = f32_to_bf16(x);
      const float rest = x - bf16_to_f32(hi);
      at[a.n * ldg] = hi;
      at[0] = f32_to_bf16(fabsf(rest) < INFINITY ? rest : 0.0f);
    } else {
      at[0] = x;
    }
  }
}

// -------------------------------------------------------------------- host

// Keys a lane for lists of `top`.
template <typename F>
void for_list(int top, F&& f) {
  if (top <= 64) f(std::integral_constant<int, 1>{});
  else if (top <= 128) f(std::integral_constant<int, 2>{});
  else if (top <= 256) f(std::integral_constant<int, 4>{});
  else if (top <= 512) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

void sort_lists(const Lists& a, int64_t n, uint32_t* keys, const Marks& marks, hipStream_t s) {
  const unsigned blocks = static_cast<unsigned>((n + 3) / 4);
  for_list(a.top, [&](auto e) {
    hipLaunchKernelGGL(k_distill_sort<decltype(e)::value>, dim3(blocks), dim3(kThreads), 0, s, a,
                       n, keys, marks);
  });
}

void store_points(const void* context, void* g, int64_t ldg, const float* c, int64_t v0, int len,
                  hipStream_t s) {
  const PointArgs& a = *static_cast<const PointArgs*>(context);
  const int64_t blocks = (a.n * a.lists.top + kThreads - 1) / kThreads;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(blocks, 1 << 16)));
  if (a.fp32)
    hipLaunchKernelGGL(k_distill_points<float>, grid, dim3(kThreads), 0, s, a,
                       static_cast<float*>(g), ldg, c, v0, len);
  else
    hipLaunchKernelGGL(k_distill_points<uint16_t>, grid, dim3(kThreads), 0, s, a,
                       static_cast<uint16_t*>(g), ldg, c, v0, len);
}

// Shares of dh's sum, which each piece of g takes: the least estimated time of
// the products (their tile core as run_dh picks it) and of the fp32 sums that
// the shares are added up in, written and read at 2.5 TB/s.  Where CUs take more
// than one tile at a time, those past 256 count up to as many on every CU: the
// one with the most decides.
// (The step, us, with the cross entropy's rule, as many shares as fill the GPU
// with 128 x 128 tiles, 16 at most, and with this one: 930 x 13715 x 5376 987 and
// 833, 2048 x 32000 x 2048 1532 and 1440, 62 x 60045 x 416 104 and 94, 122 x 55297
// x 960 180 and 158.)
int pick_splits(int64_t n, int64_t dim, int64_t piece, int32_t dtype) {
  const bool half = dtype == MUON_DTYPE_BF16;
  int best = 1;
  double least = 0.0;
  for (int s = 1; s <= kMostSplits && (s == 1 || piece / s >= 512); ++s) {
    const int64_t k = (half ? 2 : 1) * ceil_div(piece, s);
    auto time = [&](const auto& table) {
      double t = 0.0;
      for (const ShapeCost& c : table) {
        const double columns = static_cast<double>(ceil_div(dim, c.bn));
        const double tiles = dh_tiles(n, s)(c.bm) * columns;
        const double even =
            c.per_cu == 1 || tiles <= 256.0 ? tiles : std::ceil(tiles / 256.0) * 256.0;
        const double e = shape_time(c, even / columns, dim, k);
        if (t == 0.0 || e < t) t = e;
      }
      return t;
    };
    double t = half && dim % 8 == 0 ? time(kShapeNN) : half ? time(kShapeAnyBf16) : time(kShapeAnyFp32);
    if (s > 1) t += 8.0 * static_cast<double>(n * dim) * s / 2.5e6 + 4.0;
    if (s == 1 || t < least) {
      best = s;
      least = t;
    }
  }
  // k_loss_dh's shares are whole steps of 64 rows, and fewer than that can cover
  // the piece: the others would add zeros.  (The estimate does not round: with
  // rounded shares 564 x 102034 x 1280 gains 4%, 134 x 94168 x 1284 loses 15.)
  return static_cast<int>(ceil_div(piece, ceil_div(ceil_div(piece, best), 64) * 64));
}

// bf16 rows off the 16-byte grid are laid out on it, padded with zeros, where
// there are rows enough for the DMA cores to gain what the copy of the weight
// costs (us, laid out and not: backward 64 x 32000 x 2001 214 and 194, 96 218 and
// 264, 192 283 and 388, step of 8192 5750 and 13700; forward 384 x 32000 x 2001
// 150 and 109, 600 x 100003 x 777 241 and 250, 2048 x 32000 x 2001 335 and 506).
constexpr int64_t kLayForward = 512, kLayBackward = 96;
bool lay_out(int64_t n, int64_t dim, int32_t dtype, bool backward) {
  return dtype == MUON_DTYPE_BF16 && dim % 8 != 0 && n >= (backward ? kLayBackward : kLayForward);
}

// The cross entropy's workspace and, behind it, the lists'; hidden and the
// weight laid out in rows of dim elements.
struct DistillWs {
  LossWs loss;
  int64_t dim;
  size_t keys, marks, stats, hidden, weight, total;
};
DistillWs distill_ws(int64_t n, int64_t vocab, int64_t dim, int64_t top, int32_t dtype,
                     bool backward) {
  DistillWs w{};
  const bool laid = lay_out(n, dim, dtype, backward);
  w.dim = laid ? ceil_div(dim, 8) * 8 : dim;
  w.loss = loss_ws(n, vocab, w.dim, dtype, backward);
  if (backward) {
    w.loss.splits = pick_splits(n, w.dim, w.loss.piece, dtype);
    // (dh's fp32 sums stand last)
    size_t o = w.loss.part;
    if (w.loss.splits > 1 || w.loss.piece < vocab || laid)
      o += align256(static_cast<size_t>(w.loss.splits) * static_cast<size_t>(n * w.dim) * 4);
    w.loss.total = o;
  }
  const int64_t rows = backward ? n : w.loss.stats_rows;
  size_t o = align256(w.loss.total);
  auto take = [&o](size_t& at, int64_t bytes) {
    at = o;
    o += align256(static_cast<size_t>(bytes));
  };
  take(w.keys, rows * top * 4);
  if (backward) {
    take(w.marks, n * 4);
    take(w.stats, n * 8);
    w.hidden = w.loss.rows;
  } else if (laid) {
    take(w.hidden, rows * w.dim * 2);
  }
  if (laid) take(w.weight, vocab * w.dim * 2);
  w.total = o;
  return w;
}
// The weight laid out, if it has to be.
const void* laid_weight(const void* weight, int64_t vocab, int64_t dim, const DistillWs& w,
                        char* ws, hipStream_t s) {
  if (w.dim == dim) return weight;
  hipLaunchKernelGGL(k_distill_lay,
                     dim3(static_cast<unsigned>(std::min<int64_t>(ceil_div(vocab, 4), 16384))),
                     dim3(kThreads), 0, s, static_cast<const char*>(weight), vocab, dim * 2,
                     w.dim * 2, ws + w.weight);
  return ws + w.weight;
}

int check_distill(int64_t n, int64_t vocab, int64_t dim, int64_t ldh, int32_t dtype, int64_t top) {
  const int rc = check_loss(n, vocab, dim, ldh, dtype);
  if (rc != MUON_OK) return rc;
  if (top < 1 || top > kMaxTop) return set_error(MUON_ERR_BAD_SHAPE, "top must be in [1, 1024]");
  return MUON_OK;
}
int check_lists(int64_t ld_ids, int64_t ld_teacher, int64_t top, int32_t teacher_dtype,
                float temperature) {
  if (!train_dtype_ok(teacher_dtype))
    return set_error(MUON_ERR_BAD_DTYPE, "teacher must be fp32 or bf16");
  if (ld_ids < top || ld_teacher < top)
    return set_error(MUON_ERR_BAD_SHAPE, "ld_ids < top or ld_teacher < top");
  if (!(temperature >= 1e-6f && temperature <= 1e6f))
    return set_error(MUON_ERR_INVALID_ARG, "temperature must be in [1e-6, 1e6]");
  return MUON_OK;
}

Lists lists_of(const void* ids, int32_t ids_64, int64_t ld_ids, const void* teacher,
               int32_t teacher_dtype, int64_t ld_teacher, int64_t vocab, int64_t top,
               float temperature) {
  return Lists{ids, teacher, ld_ids, ld_teacher, vocab, ids_64 != 0,
               teacher_dtype == MUON_DTYPE_BF16, static_cast<int>(top), 1.0f / temperature};
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

size_t distill_loss_workspace_size(int64_t n, int64_t vocab, int64_t dim, int64_t top,
                                   int32_t dtype, int32_t backward) {
  if (n <= 0 || check_distill(n, vocab, dim, dim, dtype, top) != MUON_OK) return 0;
  const size_t forward = distill_ws(n, vocab, dim, top, dtype, false).total;
  return backward ? std::max(forward, distill_ws(n, vocab, dim, top, dtype, true).total) : forward;
}

int distill_loss_forward(const void* hidden, int64_t ld_hidden, const void* weight, int32_t dtype,
                         const void* ids, int32_t ids_64, int64_t ld_ids, const void* teacher,
                         int32_t teacher_dtype, int64_t ld_teacher, int64_t n, int64_t vocab,
                         int64_t dim, int64_t top, float temperature, float* loss, float* lse,
                         float* logp, void* workspace, size_t workspace_bytes,
                         hipStream_t stream) {
  int rc = check_distill(n, vocab, dim, ld_hidden, dtype, top);
  if (rc != MUON_OK) return rc;
  rc = check_lists(ld_ids, ld_teacher, top, teacher_dtype, temperature);
  if (rc != MUON_OK) return rc;
  if (n == 0) return MUON_OK;
  if (hidden == nullptr || weight == nullptr || ids == nullptr || teacher == nullptr ||
      loss == nullptr || lse == nullptr || logp == nullptr)
    return set_error(MUON_ERR_INVALID_ARG,
                     "hidden, weight, ids, teacher, loss, lse or logp is null");
  const DistillWs w = distill_ws(n, vocab, dim, top, dtype, false);
  if ((rc = check_ws(workspace, workspace_bytes, w.total, "distill_loss_forward")) != MUON_OK)
    return rc;
  char* ws = static_cast<char*>(workspace);
  uint32_t* keys = reinterpret_cast<uint32_t*>(ws + w.keys);
  const size_t sz = train_dtype_size(dtype), isz = ids_64 ? 8 : 4;
  const size_t zsz = train_dtype_size(teacher_dtype);
  const bool laid = w.dim != dim;
  const void* laid_w = laid_weight(weight, vocab, dim, w, ws, stream);
  for (int64_t r0 = 0; r0 < n; r0 += w.loss.stats_rows) {
    const int rows = static_cast<int>(std::min(w.loss.stats_rows, n - r0));
    const char* h = static_cast<const char*>(hidden) + static_cast<size_t>(r0 * ld_hidden) * sz;
    const Lists lists =
        lists_of(static_cast<const char*>(ids) + static_cast<size_t>(r0 * ld_ids) * isz, ids_64,
                 ld_ids, static_cast<const char*>(teacher) + static_cast<size_t>(r0 * ld_teacher) * zsz,
                 teacher_dtype, ld_teacher, vocab, top, temperature);
    Marks marks{};
    if (laid) {
      marks.hidden = h;
      marks.rows = ws + w.hidden;
      marks.stride = ld_hidden * 2;
      marks.bytes = dim * 2;
      marks.room = w.dim * 2;
    }
    sort_lists(lists, rows, keys, marks, stream);
    StatsArgs a{};
    a.h = laid ? ws + w.hidden : h;
    a.w = laid_w;
    a.tile_m = reinterpret_cast<float*>(ws + w.loss.tile_m);
    a.tile_s = reinterpret_cast<float*>(ws + w.loss.tile_s);
    a.keys = keys;
    a.points = logp + r0 * top;
    a.ldh = laid ? w.dim : ld_hidden;
    a.vocab = vocab;
    a.n = rows;
    a.dim = static_cast<int>(w.dim);
    a.top = static_cast<int>(top);
    a.scale = lists.scale;
    const int tiles = loss_stats<true>(a, dtype, stream);
    const int per = join_rows(rows);
    for_list(a.top, [&](auto e) {
      auto* kernel = per == 4 ? k_distill_join<4, decltype(e)::value>
                              : k_distill_join<16, decltype(e)::value>;
      hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>((rows + per - 1) / per)),
                         dim3(kThreads), 0, stream, a.tile_m, a.tile_s, tiles, rows, lists,
                         loss + r0, lse + r0, a.points);
    });
  }
  return check_launch("distillation loss launch");
}

int distill_loss_backward(const void* hidden, int64_t ld_hidden, const void* weight, int32_t dtype,
                          const void* ids, int32_t ids_64, int64_t ld_ids, const void* teacher,
                          int32_t teacher_dtype, int64_t ld_teacher, int64_t n, int64_t vocab,
                          int64_t dim, int64_t top, float temperature, const float* lse,
                          const float* logp, const float* dloss, void* dhidden,
                          int32_t dhidden_dtype, int64_t ld_dhidden, void* dweight,
                          int32_t dweight_dtype, int32_t accumulate, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
  int rc = check_distill(n, vocab, dim, ld_hidden, dtype, top);
  if (rc != MUON_OK) return rc;
  rc = check_lists(ld_ids, ld_teacher, top, teacher_dtype, temperature);
  if (rc != MUON_OK) return rc;
  if (dhidden != nullptr) {
    if (!train_dtype_ok(dhidden_dtype))
      return set_error(MUON_ERR_BAD_DTYPE, "dhidden must be fp32 or bf16");
    if (ld_dhidden < dim) return set_error(MUON_ERR_BAD_SHAPE, "ld_dhidden < dim");
  }
  if (dweight != nullptr && !train_dtype_ok(dweight_dtype))
    return set_error(MUON_ERR_BAD_DTYPE, "dweight must be fp32 or bf16");
  if (n == 0) return loss_no_rows(dweight, dweight_dtype, vocab, dim, accumulate, stream);
  if (dhidden == nullptr && dweight == nullptr) return MUON_OK;
  if (hidden == nullptr || weight == nullptr || ids == nullptr || teacher == nullptr ||
      lse == nullptr || logp == nullptr || dloss == nullptr)
    return set_error(MUON_ERR_INVALID_ARG,
                     "hidden, weight, ids, teacher, lse, logp or dloss is null");
  const DistillWs w = distill_ws(n, vocab, dim, top, dtype, true);
  if ((rc = check_ws(workspace, workspace_bytes, w.total, "distill_loss_backward")) != MUON_OK)
    return rc;
  char* ws = static_cast<char*>(workspace);
  uint32_t* keys = reinterpret_cast<uint32_t*>(ws + w.keys);
  int32_t* marks = reinterpret_cast<int32_t*>(ws + w.marks);
  f32x2_t* stats = reinterpret_cast<f32x2_t*>(ws + w.stats);
  const int64_t sz = static_cast<int64_t>(train_dtype_size(dtype));
  const Lists lists = lists_of(ids, ids_64, ld_ids, teacher, teacher_dtype, ld_teacher, vocab, top,
                               temperature);
  const bool laid = w.dim != dim;
  sort_lists(lists, n, keys,
             Marks{marks, stats, static_cast<const char*>(hidden),
                   dweight != nullptr || laid ? ws + w.hidden : nullptr, ld_hidden * sz, dim * sz,
                   w.dim * sz},
             stream);
  const PointArgs points{lists, keys, stats, logp, dloss, n, dtype == MUON_DTYPE_FP32};
  BackwardArgs b{};
  // (a row without a list has no gradient: its zeros will do)
  b.h = laid ? ws + w.hidden : static_cast<const char*>(hidden);
  b.w = laid_weight(weight, vocab, dim, w, ws, stream);
  b.targets = marks;  // rows with a list; the marked column is stored again
  b.lse = lse;
  b.dloss = dloss;
  b.dh = dhidden;
  b.dw = dweight;
  b.n = n;
  b.vocab = vocab;
  b.dim = w.dim;
  b.ldh = laid ? w.dim : ld_hidden;
  b.ld_dh = ld_dhidden;
  b.cols = dim;
  b.accumulate = accumulate != 0;
  b.ws = ws;
  b.scale = lists.scale;
  b.after_g = store_points;
  b.context = &points;
  loss_backward<true>(b, w.loss, dtype, dhidden_dtype, dweight_dtype, stream);
  return check_launch("distillation loss gradient launch");
}

}  // extern "C"
