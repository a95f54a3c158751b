// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out[t]   = scale * E[id_t]
//   dE[v]    = scale * sum over t with id_t = v of dout[t]    (+ dE[v])
//
// Both are bound by HBM: the lookup reads the rows its positions name and
// writes n rows, the gradient reads n rows and writes the whole dense
// table gradient, which the optimizer step reads next.
//
// The gradient sorts the positions by id (stable, so that every sum runs in
// the order of the positions and repeated calls give the same bits), cuts
// the sorted list into chunks of 16 or 32 positions and sums each run of
// equal ids inside a chunk in fp32 registers.  A run that lies inside its
// chunk is finished there; a run that crosses a chunk border leaves one
// fp32 partial row per chunk, which a second kernel adds in chunk order.
// A frequent token therefore spreads over as many workgroups as a rare one.
//
// Rows that no position names are zeroed by workgroups of their own: the
// first rows beside the sort, which leaves the GPU idle (whether named or
// not), the rest beside the sums, when the sorted ids tell which they are.
#include <algorithm>
#include <cmath>

#include "train_common.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = kThreads * 8;  // columns per workgroup, 8 per thread

// ------------------------------------------------------------------ lookup

// One workgroup: kRows positions x kCols columns; the loads of all its rows
// are in flight together.
constexpr int kRows = 4;

template <bool STREAM, typename TT, typename TO, typename ID>
__global__ __launch_bounds__(kThreads) void k_embed_fwd(const TT* __restrict__ table,
                                                        const ID* __restrict__ ids, int64_t n,
                                                        int64_t vocab, int64_t dim, float scale,
                                                        TO* __restrict__ out, int64_t ld) {
  const int64_t c = static_cast<int64_t>(blockIdx.y) * kCols + threadIdx.x * 8;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows;
  if (c >= dim) return;
  int64_t id[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int64_t v = t0 + r < n ? static_cast<int64_t>(ids[t0 + r]) : -1;
    id[r] = v >= 0 && v < vocab ? v : -1;
  }
  if (c + 8 <= dim) {
    float x[kRows][8];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[r][k] = 0.0f;
      if (id[r] >= 0) load8(table + id[r] * dim + c, x[r]);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (t0 + r >= n) break;
#pragma unroll
      for (int k = 0; k < 8; ++k) x[r][k] *= scale;
      if (id[r] < 0) {  // no row: zeros also where scale is not finite
#pragma unroll
        for (int k = 0; k < 8; ++k) x[r][k] = 0.0f;
      }
      store8<STREAM>(out + (t0 + r) * ld + c, x[r]);
    }
  } else {
    for (int r = 0; r < kRows && t0 + r < n; ++r)
      for (int64_t j = c; j < dim; ++j) {
        const float v = id[r] >= 0 ? to_f32(table[id[r] * dim + j]) * scale : 0.0f;
        from_f32(v, out + (t0 + r) * ld + j);
      }
  }
}

// -------------------------------------------------------------------- sort
//
// Stable sort of (key, position) by key: key = id, or vocab for an id outside
// [0, vocab), which puts the positions without a row last.
//
// Up to kRankN keys: a key's place is the number of keys that are smaller,
// or equal and before it.  All pairs are compared, n^2 / 64 wave
// instructions spread over the GPU, in one launch (one workgroup's radix
// sort of 8192 keys in LDS took 26 us).
// More: LSD radix sort, at most kMaxBits bits a pass, a histogram and a
// scatter launch each.  Each wave owns a contiguous part of its workgroup's
// keys and places 64 keys at a time, a key's rank among equal digits of the
// 64 being the number of lower lanes that hold the digit.

constexpr int kMaxBits = 9;
constexpr int kMaxBins = 1 << kMaxBits;

__device__ __forceinline__ uint32_t clip_key(int64_t v, int64_t vocab) {
  return static_cast<uint32_t>(v >= 0 && v < vocab ? v : vocab);
}

// lanes of the wave (among `active`) whose digit equals this lane's
__device__ __forceinline__ uint64_t match_digit(uint32_t d, int bits, uint64_t active) {
  uint64_t m = active;
  for (int b = 0; b < bits; ++b) {
    const uint64_t vote = __ballot((d >> b) & 1u);
    m &= ((d >> b) & 1u) ? vote : ~vote;
  }
  return m;
}

// Exclusive scan of h[0..n) in LDS by the whole workgroup (T threads,
// n <= 2T); tmp: T / 64 entries.
template <int T>
__device__ __forceinline__ void block_exclusive_scan(uint32_t* h, int n, uint32_t* tmp) {
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const uint32_t a = 2 * t < n ? h[2 * t] : 0, b = 2 * t + 1 < n ? h[2 * t + 1] : 0;
  uint32_t s = a + b;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t u = __shfl_up(s, o, 64);
    if (lane >= o) s += u;
  }
  if (lane == 63) tmp[w] = s;
  __syncthreads();
  uint32_t base = 0;
  for (int k = 0; k < w; ++k) base += tmp[k];
  const uint32_t ex = base + s - (a + b);
  if (2 * t < n) h[2 * t] = ex;
  if (2 * t + 1 < n) h[2 * t + 1] = ex + a;
  __syncthreads();
}

// Zeroes n elements from g: the part of workgroup `b` of `nb`.
template <typename TG>
__device__ __forceinline__ void zero_part(TG* g, int64_t n, int64_t b, int64_t nb, int threads) {
  // 16-byte stores on the aligned middle, the ragged ends by workgroup 0
  const int64_t per = 16 / sizeof(TG);
  const int64_t mis = static_cast<int64_t>((reinterpret_cast<uintptr_t>(g) & 15) / sizeof(TG));
  int64_t head = mis ? per - mis : 0;
  if (head > n) head = n;
  const int64_t n16 = (n - head) / per;
  u32x4_t* v = reinterpret_cast<u32x4_t*>(g + head);
  for (int64_t i = b * threads + threadIdx.x; i < n16; i += nb * threads) v[i] = u32x4_t{0, 0, 0, 0};
  if (b == 0) {
    if (static_cast<int64_t>(threadIdx.x) < head) g[threadIdx.x] = TG{};
    const int64_t t = head + n16 * per + threadIdx.x;
    if (t < n) g[t] = TG{};
  }
}
// Zeroes the rows of [r0, r0 + 32) whose bit of `named` is clear and that
// are below vocab: part `b` of `nb`.
template <typename TG>
__device__ __forceinline__ void zero_rows(TG* g, uint32_t named, int64_t r0, int64_t vocab,
                                          int64_t dim, int b, int nb, int threads) {
  const int rows = static_cast<int>(vocab - r0 < 32 ? vocab - r0 : 32);
  for (int r = 0; r < rows;) {
    if ((named >> r) & 1u) {
      ++r;
      continue;
    }
    int e = r + 1;
    while (e < rows && !((named >> e) & 1u)) ++e;
    zero_part(g + (r0 + r) * dim, (e - r) * dim, b, nb, threads);
    r = e;
  }
}

// Zeroes the rows from v0 on that are not among the sorted keys.  Workgroup
// b takes part b % parts of every so many-th group of 32 rows; lane l of
// each wave looks row l of the group up.
template <typename TG>
__device__ __forceinline__ void zero_unnamed(TG* g, const uint32_t* keys, int64_t n, int64_t v0,
                                             int64_t vocab, int64_t dim, int64_t b, int64_t nb,
                                             int parts, int threads) {
  const int lane = threadIdx.x & 63;
  for (int64_t r0 = v0 + b / parts * 32; r0 < vocab; r0 += nb / parts * 32) {
    bool named = false;
    if (lane < 32 && r0 + lane < vocab) {
      const uint32_t row = static_cast<uint32_t>(r0 + lane);
      int64_t lo = 0, hi = n;
      while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (keys[mid] < row) lo = mid + 1;
        else hi = mid;
      }
      named = lo < n && keys[lo] == row;
    }
    zero_rows(g, static_cast<uint32_t>(__ballot(named)), r0, vocab, dim,
              static_cast<int>(b % parts), parts, threads);
  }
}

constexpr int kRankN = 16384;
constexpr int kRankThreads = 1024;
constexpr int kRankWaves = kRankThreads / 64;

// Each workgroup places 64 keys, one a lane; its waves share the keys they
// are compared with.  The workgroups from rank_blocks on zero the first
// zero_n elements of the table gradient.
template <typename ID, typename TG>
__global__ __launch_bounds__(kRankThreads) void k_sort_rank(
    const ID* __restrict__ ids, int n, int64_t vocab, int rank_blocks,
    uint32_t* __restrict__ keys_out, uint32_t* __restrict__ pos_out, TG* __restrict__ dtable,
    int64_t zero_n) {
  __shared__ __attribute__((aligned(16))) uint32_t key[kRankN];
  __shared__ uint32_t red[kRankWaves][64];
  if (static_cast<int>(blockIdx.x) >= rank_blocks) {
    zero_part(dtable, zero_n, blockIdx.x - rank_blocks, gridDim.x - rank_blocks, kRankThreads);
    return;
  }
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  // padded to whole groups of 64 with a key above all others
  const int np = (n + 63) / 64 * 64;
  for (int i = t; i < np; i += kRankThreads)
    key[i] = i < n ? clip_key(static_cast<int64_t>(ids[i]), vocab) : 0xffffffffu;
  __syncthreads();
  const int i0 = blockIdx.x * 64, i = i0 + lane;
  const uint32_t ki = key[i];
  uint32_t count = 0;
  // keys of [lo, hi) below x, both multiples of 4
  auto below = [&](int lo, int hi, uint32_t x) {
#pragma unroll 8
    for (int j = lo; j < hi; j += 4) {
      const uint4 k = *reinterpret_cast<const uint4*>(key + j);
      count += k.x < x;
      count += k.y < x;
      count += k.z < x;
      count += k.w < x;
    }
  };
  // this wave's part; equal keys count where they come before, so k <= ki,
  // that is k < ki + 1, in the groups of 64 before this one (a position of
  // the padding is not placed: its ki + 1 may wrap)
  const int part = (np / 64 + kRankWaves - 1) / kRankWaves * 64;
  const int lo = min(w * part, np), hi = min(lo + part, np);
  below(lo, min(hi, i0), ki + 1u);
  below(max(lo, i0 + 64), hi, ki);
  if (lo <= i0 && i0 < hi)
    for (int j = 0; j < 64; ++j) {
      const uint32_t k = key[i0 + j];
      count += k < ki || (k == ki && j < lane);
    }
  red[w][lane] = count;
  __syncthreads();
  if (w != 0 || i >= n) return;
  uint32_t rank = 0;
#pragma unroll
  for (int k = 0; k < kRankWaves; ++k) rank += red[k][lane];
  keys_out[rank] = ki;
  pos_out[rank] = static_cast<uint32_t>(i);
}

// Radix passes: at most kSortBlocks workgroups, so that each can add up the
// others' histograms by itself; part: keys of a wave, a multiple of 64.
constexpr int kSortThreads = 256;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortBlocks = 64;

// The first pass reads the ids themselves (FIRST); its launch has more
// workgroups, which zero the first zero_n elements of the table gradient.
template <bool FIRST, typename ID, typename TG>
__global__ __launch_bounds__(kSortThreads) void k_sort_hist(
    const ID* __restrict__ ids, const uint32_t* __restrict__ keys, int64_t n, int64_t vocab,
    int shift, int bits, int n_blocks, int part, uint32_t* __restrict__ hist,
    TG* __restrict__ dtable, int64_t zero_n) {
  if (FIRST && static_cast<int>(blockIdx.x) >= n_blocks) {
    zero_part(dtable, zero_n, blockIdx.x - n_blocks, gridDim.x - n_blocks, kSortThreads);
    return;
  }
  __shared__ uint32_t cnt[kMaxBins];
  const int bins = 1 << bits;
  for (int b = threadIdx.x; b < bins; b += kSortThreads) cnt[b] = 0;
  __syncthreads();
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * part * kSortWaves;
  for (int k = threadIdx.x; k < part * kSortWaves && i0 + k < n; k += kSortThreads) {
    const uint32_t key = FIRST ? clip_key(static_cast<int64_t>(ids[i0 + k]), vocab) : keys[i0 + k];
    atomicAdd(&cnt[(key >> shift) & (bins - 1)], 1u);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads)
    hist[static_cast<int64_t>(blockIdx.x) * bins + b] = cnt[b];
}

template <bool FIRST, typename ID>
__global__ __launch_bounds__(kSortThreads) void k_sort_scatter(
    const ID* __restrict__ ids, const uint32_t* __restrict__ keys,
    const uint32_t* __restrict__ pos, int64_t n, int64_t vocab, int shift, int bits, int n_blocks,
    int part, const uint32_t* __restrict__ hist, uint32_t* __restrict__ keys_out,
    uint32_t* __restrict__ pos_out) {
  __shared__ uint32_t cnt[kSortWaves][kMaxBins];
  __shared__ uint32_t base[kMaxBins], tmp[kSortWaves];
  const int bins = 1 << bits;
  const uint32_t mask = static_cast<uint32_t>(bins) - 1u;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  for (int i = t; i < kSortWaves * kMaxBins; i += kSortThreads) cnt[0][i] = 0;
  __syncthreads();
  const int64_t lo = (static_cast<int64_t>(blockIdx.x) * kSortWaves + w) * part;
  const int64_t hi = lo + part < n ? lo + part : n;
  auto key_at = [&](int64_t i) {
    return FIRST ? clip_key(static_cast<int64_t>(ids[i]), vocab) : keys[i];
  };
  for (int64_t i = lo + lane; i < hi; i += 64) atomicAdd(&cnt[w][(key_at(i) >> shift) & mask], 1u);
  // a digit's first place: all keys with lower digits, then this digit's in
  // the workgroups before this one, then in this one's waves before
  uint32_t before[kMaxBins / kSortThreads];
#pragma unroll
  for (int u = 0; u < kMaxBins / kSortThreads; ++u) {
    const int b = t + u * kSortThreads;
    before[u] = 0;
    if (b < bins) {
      uint32_t all = 0;
#pragma unroll 8
      for (int k = 0; k < n_blocks; ++k) {
        const uint32_t c = hist[static_cast<int64_t>(k) * bins + b];
        all += c;
        if (k < static_cast<int>(blockIdx.x)) before[u] += c;
      }
      base[b] = all;
    }
  }
  __syncthreads();
  block_exclusive_scan<kSortThreads>(base, bins, tmp);
#pragma unroll
  for (int u = 0; u < kMaxBins / kSortThreads; ++u) {
    const int b = t + u * kSortThreads;
    if (b < bins) {
      uint32_t s = base[b] + before[u];
      for (int j = 0; j < kSortWaves; ++j) {
        const uint32_t c = cnt[j][b];
        cnt[j][b] = s;
        s += c;
      }
    }
  }
  __syncthreads();
  for (int64_t i0 = lo; i0 < hi; i0 += 64) {
    const int64_t i = i0 + lane;
    const bool on = i < hi;
    const uint32_t k = on ? key_at(i) : 0u;
    const uint32_t d = (k >> shift) & mask;
    const uint64_t m = match_digit(d, bits, __ballot(on));
    if (on) {
      const uint32_t to = cnt[w][d] + __popcll(m & ((1ull << lane) - 1ull));
      keys_out[to] = k;
      pos_out[to] = FIRST ? static_cast<uint32_t>(i) : pos[i];
      // the last lane of the digit moves the wave's counter on
      if ((m >> lane) == 1ull) cnt[w][d] += __popcll(m);
    }
    wave_sync();  // the wave's next 64 keys read the counters just moved
  }
}

// -------------------------------------------------------------------- sums

constexpr int kSumThreads = 128;
constexpr int kSumCols = kSumThreads * 8;

// The row of a finished run: scale * sum, plus the old row when
// accumulating; cols columns (1..8) from c.
template <typename TG>
__device__ __forceinline__ void write_row(TG* p, float* acc, int cols, float scale,
                                          int accumulate) {
  if (cols == 8) {
    float o[8];
    if (accumulate) {
      load8(p, o);
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = fmaf(scale, acc[k], o[k]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = scale * acc[k];
    }
    store8(p, o);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < cols)
        from_f32(accumulate ? fmaf(scale, acc[k], to_f32(p[k])) : scale * acc[k], p + k);
  }
}

// Partial rows: slot 0 of a chunk holds the run that continues from the
// chunk before, slot 1 the one that starts in it and runs on.  dim_p: dim
// rounded up to 8, so that every partial access is whole and aligned.
__device__ __forceinline__ float* partial_row(float* parts, int64_t chunk, int slot,
                                              int64_t dim_p) {
  return parts + (2 * chunk + slot) * dim_p;
}

// The workgroups from sum_blocks on zero the unnamed rows from zero_v0 on.
template <typename TD, typename TG>
__global__ __launch_bounds__(kSumThreads) void k_embed_runs(
    const TD* __restrict__ dout, int64_t ld, const uint32_t* __restrict__ keys,
    const uint32_t* __restrict__ pos, int64_t n, int64_t vocab, int64_t dim, int64_t dim_p,
    int chunk_len, float scale, int accumulate, TG* __restrict__ dtable,
    float* __restrict__ parts, int64_t sum_blocks, int slices, int64_t zero_v0,
    int zero_parts) {
  if (static_cast<int64_t>(blockIdx.x) >= sum_blocks) {
    zero_unnamed(dtable, keys, n, zero_v0, vocab, dim, blockIdx.x - sum_blocks,
                 gridDim.x - sum_blocks, zero_parts, kSumThreads);
    return;
  }
  const int64_t chunk = blockIdx.x / slices;
  const int64_t s0 = chunk * chunk_len;
  const int len = static_cast<int>(n - s0 < chunk_len ? n - s0 : chunk_len);
  const int64_t c = static_cast<int64_t>(blockIdx.x % slices) * kSumCols + threadIdx.x * 8;
  if (c >= dim) return;
  const int cols = static_cast<int>(dim - c < 8 ? dim - c : 8);
  const uint32_t none = static_cast<uint32_t>(vocab);
  const uint32_t before = s0 > 0 ? keys[s0 - 1] : none;
  const uint32_t after = s0 + len < n ? keys[s0 + len] : none;
  float acc[8] = {};
  bool first = true;  // still in the chunk's first run
  constexpr int U = 8;
  for (int i0 = 0; i0 < len; i0 += U) {
    float x[U][8];
    uint32_t key[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      key[u] = none;
#pragma unroll
      for (int k = 0; k < 8; ++k) x[u][k] = 0.0f;
      if (i0 + u >= len) continue;
      key[u] = keys[s0 + i0 + u];
      if (key[u] == none) continue;
      const TD* p = dout + static_cast<int64_t>(pos[s0 + i0 + u]) * ld + c;
      if (cols == 8) {
        load8(p, x[u]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < cols) x[u][k] = to_f32(p[k]);
      }
    }
    // the key after the last of this batch
    uint32_t next = i0 + U < len ? keys[s0 + i0 + U] : after;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (key[u] == none) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] += x[u][k];
      const int i = i0 + u;
      const uint32_t nk = u + 1 < U ? (i + 1 < len ? key[u + 1] : after) : next;
      const bool last = i + 1 == len;
      if (nk == key[u] && !last) continue;
      const bool head = first && before == key[u];
      const bool tail = last && after == key[u];
      if (head || tail) {
        store8(partial_row(parts, chunk, head ? 0 : 1, dim_p) + c, acc);
      } else {
        write_row(dtable + static_cast<int64_t>(key[u]) * dim + c, acc, cols, scale, accumulate);
      }
      first = false;
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = 0.0f;
    }
  }
}

// Adds the partial rows of the run that starts in this chunk and crosses
// its end, in chunk order.
template <typename TG>
__global__ __launch_bounds__(kSumThreads) void k_embed_join(
    const uint32_t* __restrict__ keys, int64_t n, int64_t vocab, int64_t dim, int64_t dim_p,
    int chunk_len, float scale, int accumulate, TG* __restrict__ dtable, float* parts,
    int slices) {
  const int64_t chunk = blockIdx.x / slices;
  const int64_t end = (chunk + 1) * chunk_len;
  if (end >= n) return;
  const uint32_t key = keys[end - 1];
  if (key == static_cast<uint32_t>(vocab) || keys[end] != key) return;
  // the run started in an earlier chunk: that chunk joins it
  if (chunk > 0 && keys[end - chunk_len] == key && keys[end - chunk_len - 1] == key) return;
  const int64_t c = static_cast<int64_t>(blockIdx.x % slices) * kSumCols + threadIdx.x * 8;
  if (c >= dim) return;
  // the last chunk that the run reaches: first position whose key exceeds it
  int64_t lo = end, hi = n;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (keys[mid] <= key) lo = mid + 1;
    else hi = mid;
  }
  const int64_t last = (lo - 1) / chunk_len;
  float acc[8];
  load8(partial_row(parts, chunk, 1, dim_p) + c, acc);
  int64_t k = chunk + 1;
  constexpr int U = 8;
  for (; k + U - 1 <= last; k += U) {
    float x[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) load8(partial_row(parts, k + u, 0, dim_p) + c, x[u]);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += x[u][e];
  }
  for (; k <= last; ++k) {
    float x[8];
    load8(partial_row(parts, k, 0, dim_p) + c, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += x[e];
  }
  write_row(dtable + static_cast<int64_t>(key) * dim + c, acc,
            static_cast<int>(dim - c < 8 ? dim - c : 8), scale, accumulate);
}

// ------------------------------------------------------------ few positions
//
// Up to kDirectN positions need no sort: the workgroup of a position compares
// its id with all others and, if it is the first to name its row, adds the
// row's positions up in order.  Other workgroups zero the rows that nobody
// names, whose bits they gather from the ids.  One launch instead of three:
// 512 positions into 32000 x 2048 take 26 us, 700 take 30, where the sort's
// three launches take 31; 1024 take 39 and 32.
constexpr int kDirectN = 640;
constexpr int kDirectRows = 4096;  // rows of a zeroing workgroup at most

template <typename TD, typename TG, typename ID>
__global__ __launch_bounds__(kSumThreads) void k_embed_direct(
    const TD* __restrict__ dout, int64_t ld, const ID* __restrict__ ids, int n, int64_t vocab,
    int64_t dim, float scale, int accumulate, TG* __restrict__ dtable, int sum_blocks, int slices,
    int zero_len, int zero_parts) {
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  if (static_cast<int>(blockIdx.x) >= sum_blocks) {
    // rows [r0, r0 + zero_len), a multiple of 32
    __shared__ uint32_t bits[kDirectRows / 32];
    const int b = blockIdx.x - sum_blocks;
    const int64_t r0 = static_cast<int64_t>(b / zero_parts) * zero_len;
    for (int i = t; i < zero_len / 32; i += kSumThreads) bits[i] = 0u;
    __syncthreads();
    for (int i = t; i < n; i += kSumThreads) {
      const int64_t id = static_cast<int64_t>(ids[i]);
      if (id < r0 || id >= r0 + zero_len) continue;
      const int v = static_cast<int>(id - r0);
      atomicOr(&bits[v >> 5], 1u << (v & 31));
    }
    __syncthreads();
    for (int i = 0; i < zero_len / 32 && r0 + 32 * i < vocab; ++i)
      zero_rows(dtable, bits[i], r0 + 32 * i, vocab, dim, b % zero_parts, zero_parts, kSumThreads);
    return;
  }
  __shared__ uint64_t same[kDirectN / 64];
  const int at = blockIdx.x / slices;
  const int64_t id = static_cast<int64_t>(ids[at]);
  if (id < 0 || id >= vocab) return;
  const int words = (n + 63) / 64;
  for (int k = w; k < words; k += kSumThreads / 64) {
    const int i = 64 * k + lane;
    const uint64_t m = __ballot(i < n && static_cast<int64_t>(ids[i]) == id);
    if (lane == 0) same[k] = m;
  }
  __syncthreads();
  // a position before this one names the row: that one's workgroup adds up
  for (int k = 0; k < at / 64; ++k)
    if (same[k] != 0) return;
  if ((same[at / 64] & ((1ull << (at % 64)) - 1ull)) != 0) return;
  const int64_t c = static_cast<int64_t>(blockIdx.x % slices) * kSumCols + t * 8;
  if (c >= dim) return;
  const int cols = static_cast<int>(dim - c < 8 ? dim - c : 8);
  float acc[8] = {};
  constexpr int U = 8;
  int k = at / 64;
  uint64_t m = same[k];
  bool more = true;
  while (more) {
    float x[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[u][e] = 0.0f;
      while (m == 0 && k + 1 < words) m = same[++k];
      more = m != 0;
      if (!more) continue;
      const int i = 64 * k + __ffsll(static_cast<unsigned long long>(m)) - 1;
      m &= m - 1;
      const TD* p = dout + i * ld + c;
      if (cols == 8) {
        load8(p, x[u]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < cols) x[u][e] = to_f32(p[e]);
      }
    }
    // (the slots left over add zeros)
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += x[u][e];
  }
  write_row(dtable + id * dim + c, acc, cols, scale, accumulate);
}

// -------------------------------------------------------------------- host

int key_bits(int64_t vocab) {
  int b = 1;
  while ((static_cast<int64_t>(1) << b) <= vocab) ++b;  // the largest key is vocab
  return b;
}

struct EmbedWs {
  size_t keys[2], pos[2], hist, parts, total;
  int64_t chunks, dim_p;
  int blocks, part;  // radix workgroups, keys of a wave
  int chunk_len, slices;
};
EmbedWs embed_ws(int64_t n, int64_t dim) {
  EmbedWs w{};
  const int64_t groups = (n + 63) / 64;  // of 64 keys; at least 4 a wave
  w.part = static_cast<int>(std::max<int64_t>(4, (groups + kSortBlocks * kSortWaves - 1) /
                                                     (kSortBlocks * kSortWaves)) * 64);
  w.blocks = static_cast<int>((n + w.part * kSortWaves - 1) / (w.part * kSortWaves));
  w.slices = static_cast<int>((dim + kSumCols - 1) / kSumCols);
  // 32 positions a chunk, or 16 where that leaves too few workgroups for the
  // 256 CUs to hide the loads' latency (8191 x 2048: 21 us against 16)
  w.chunk_len = (n + 31) / 32 * w.slices >= 4096 ? 32 : 16;
  w.chunks = (n + w.chunk_len - 1) / w.chunk_len;
  w.dim_p = (dim + 7) / 8 * 8;
  size_t o = 0;
  for (int k = 0; k < 2; ++k) {
    w.keys[k] = o;
    o += align256(static_cast<size_t>(n) * 4);
    w.pos[k] = o;
    o += align256(static_cast<size_t>(n) * 4);
  }
  w.hist = o;
  o += align256(static_cast<size_t>(w.blocks) * kMaxBins * 4);
  w.parts = o;
  o += static_cast<size_t>(w.chunks) * 2 * static_cast<size_t>(w.dim_p) * 4;
  w.total = o;
  return w;
}

int check_sizes(int64_t n, int64_t vocab, int64_t dim, float scale) {
  const int rc = check_token_sizes(n, vocab, dim);
  if (rc != MUON_OK) return rc;
  if (!std::isfinite(scale)) return set_error(MUON_ERR_INVALID_ARG, "scale must be finite");
  return MUON_OK;
}

// Outputs of which the last-level cache (256 MiB) would keep little.
constexpr int64_t kStreamBytes = int64_t{320} << 20;

template <typename TT, typename TO, typename ID>
void run_fwd(const void* table, const void* ids, int64_t n, int64_t vocab, int64_t dim,
             float scale, void* out, int64_t ld, hipStream_t s) {
  // A large output is stored past the caches, if its rows are whole lines:
  // 32768 x 7168 in 108 us against 135, and with a pass that reads it 271
  // against 285; 24576 x 7168 82 and 202 against 102 and 205.  From smaller ones
  // the reader loses what the lookup gains: 20000 x 7168 (273 MiB) 68 and 164
  // against 83 and 158.
  const int64_t sz = static_cast<int64_t>(sizeof(TO));
  const bool stream = n * dim * sz >= kStreamBytes && reinterpret_cast<uintptr_t>(out) % 128 == 0 &&
                      ld * sz % 128 == 0 && dim * sz % 128 == 0;
  auto* kernel = stream ? k_embed_fwd<true, TT, TO, ID> : k_embed_fwd<false, TT, TO, ID>;
  // a launch holds fewer than 2^32 threads along x
  constexpr int64_t kMost = int64_t{1} << 25;
  const unsigned ny = static_cast<unsigned>((dim + kCols - 1) / kCols);
  for (int64_t t0 = 0; t0 < n; t0 += kMost) {
    const int64_t m = std::min(n - t0, kMost);
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>((m + kRows - 1) / kRows), ny),
                       dim3(kThreads), 0, s, static_cast<const TT*>(table),
                       static_cast<const ID*>(ids) + t0, m, vocab, dim, scale,
                       static_cast<TO*>(out) + t0 * ld, ld);
  }
}

// Workgroups that zero `bytes`: enough to reach the write rate, few enough
// that each has several stores.
int zero_blocks(int64_t bytes, int threads) {
  const int64_t pieces = (bytes + 64 * threads - 1) / (64 * threads);
  return static_cast<int>(pieces < 4096 ? pieces : 4096);
}
// Workgroups to a group of rows that are zeroed, for 2048 in all.
int zero_parts(int64_t groups) {
  return groups <= 0 ? 1 : static_cast<int>(std::max<int64_t>(1, 2048 / groups));
}
// Bytes zeroed beside the sort: about what its time allows.  (4096 positions
// into 32000 x 2048: 42 us with 32 MiB, 34 with 64, 36 with 128; 8191: 46, 46
// and 39.)
int64_t zero_with_sort(int64_t n) {
  return std::min<int64_t>(int64_t{128} << 20, std::max<int64_t>(int64_t{32} << 20, n << 14));
}

struct BackwardArgs {
  const void *dout, *ids;
  int64_t ld, n, vocab, dim;
  float scale;
  void* dtable;
  int accumulate;
  char* ws;
};

template <typename TD, typename TG, typename ID>
void run_backward(const BackwardArgs& a, const EmbedWs& w, hipStream_t s) {
  const ID* ids = static_cast<const ID*>(a.ids);
  TG* dt = static_cast<TG*>(a.dtable);
  const int64_t n = a.n, vocab = a.vocab;
  if (n > 0 && n <= kDirectN) {
    const int sum_blocks = static_cast<int>(n) * w.slices;
    // groups of rows for the zeroing workgroups: 32, more for a table of very
    // many rows; several workgroups to a group where there are few
    const int64_t len = std::min<int64_t>(kDirectRows, ((vocab + 4095) / 4096 + 31) / 32 * 32);
    const int64_t groups = a.accumulate ? 0 : (vocab + len - 1) / len;
    const int parts = zero_parts(groups);
    hipLaunchKernelGGL((k_embed_direct<TD, TG, ID>),
                       dim3(static_cast<unsigned>(sum_blocks + groups * parts)), dim3(kSumThreads),
                       0, s, static_cast<const TD*>(a.dout), a.ld, ids, static_cast<int>(n), vocab,
                       a.dim, a.scale, a.accumulate, dt, sum_blocks, w.slices,
                       static_cast<int>(len), parts);
    return;
  }
  // rows [0, zero_v0) are zeroed before the sums
  const int64_t row_bytes = a.dim * static_cast<int64_t>(sizeof(TG));
  int64_t zero_v0 = a.accumulate ? vocab : zero_with_sort(n) / row_bytes;
  if (zero_v0 > vocab || n == 0) zero_v0 = vocab;
  const int64_t zero_n = a.accumulate ? 0 : zero_v0 * a.dim;
  const int64_t zero_bytes = zero_n * static_cast<int64_t>(sizeof(TG));
  if (n == 0) {
    hipLaunchKernelGGL((k_sort_rank<ID, TG>), dim3(zero_blocks(zero_bytes, kRankThreads)),
                       dim3(kRankThreads), 0, s, ids, 0, vocab, 0, nullptr, nullptr, dt, zero_n);
    return;
  }
  uint32_t* keys[2] = {reinterpret_cast<uint32_t*>(a.ws + w.keys[0]),
                       reinterpret_cast<uint32_t*>(a.ws + w.keys[1])};
  uint32_t* pos[2] = {reinterpret_cast<uint32_t*>(a.ws + w.pos[0]),
                      reinterpret_cast<uint32_t*>(a.ws + w.pos[1])};
  uint32_t* hist = reinterpret_cast<uint32_t*>(a.ws + w.hist);
  int cur = 0;
  if (n <= kRankN) {
    const int rb = static_cast<int>((n + 63) / 64);
    hipLaunchKernelGGL((k_sort_rank<ID, TG>), dim3(rb + zero_blocks(zero_bytes, kRankThreads)),
                       dim3(kRankThreads), 0, s, ids, static_cast<int>(n), vocab, rb, keys[0],
                       pos[0], dt, zero_n);
  } else {
    const int all = key_bits(vocab);
    const int passes = (all + kMaxBits - 1) / kMaxBits;
    const int bits = (all + passes - 1) / passes;
    const dim3 grid(w.blocks), block(kSortThreads);
    for (int p = 0; p < passes; ++p) {
      const int shift = p * bits;
      if (p == 0) {
        hipLaunchKernelGGL((k_sort_hist<true, ID, TG>),
                           dim3(w.blocks + zero_blocks(zero_bytes, kSortThreads)), block, 0, s, ids,
                           nullptr, n, vocab, shift, bits, w.blocks, w.part, hist, dt, zero_n);
        hipLaunchKernelGGL((k_sort_scatter<true, ID>), grid, block, 0, s, ids, nullptr, nullptr, n,
                           vocab, shift, bits, w.blocks, w.part, hist, keys[1], pos[1]);
      } else {
        hipLaunchKernelGGL((k_sort_hist<false, ID, TG>), grid, block, 0, s, ids, keys[cur], n,
                           vocab, shift, bits, w.blocks, w.part, hist, dt, int64_t{0});
        hipLaunchKernelGGL((k_sort_scatter<false, ID>), grid, block, 0, s, ids, keys[cur],
                           pos[cur], n, vocab, shift, bits, w.blocks, w.part, hist, keys[cur ^ 1],
                           pos[cur ^ 1]);
      }
      cur ^= 1;
    }
  }
  const int64_t sum_blocks = w.chunks * w.slices;
  const int64_t groups = (vocab - zero_v0 + 31) / 32;
  const int zparts = zero_parts(groups);
  const int64_t zb = std::min<int64_t>(groups, 4096) * zparts;
  float* parts = reinterpret_cast<float*>(a.ws + w.parts);
  hipLaunchKernelGGL((k_embed_runs<TD, TG>), dim3(static_cast<unsigned>(sum_blocks + zb)),
                     dim3(kSumThreads), 0, s, static_cast<const TD*>(a.dout), a.ld, keys[cur],
                     pos[cur], n, vocab, a.dim, w.dim_p, w.chunk_len, a.scale, a.accumulate, dt,
                     parts, sum_blocks, w.slices, zero_v0, zparts);
  if (w.chunks > 1)
    hipLaunchKernelGGL(k_embed_join<TG>, dim3(static_cast<unsigned>(sum_blocks)),
                       dim3(kSumThreads), 0, s, keys[cur], n, vocab, a.dim, w.dim_p, w.chunk_len,
                       a.scale, a.accumulate, dt, parts, w.slices);
}

template <typename TD, typename TG>
void run_backward(const BackwardArgs& a, const EmbedWs& w, bool ids_64, hipStream_t s) {
  if (ids_64) run_backward<TD, TG, int64_t>(a, w, s);
  else run_backward<TD, TG, int32_t>(a, w, s);
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

int embed_forward(const void* table, int32_t table_dtype, int64_t vocab, int64_t dim,
                  const void* ids, int32_t ids_64, int64_t n, float scale, void* out,
                  int32_t out_dtype, int64_t ld_out, hipStream_t stream) {
  const int rc = check_sizes(n, vocab, dim, scale);
  if (rc != MUON_OK) return rc;
  if (!train_dtype_ok(table_dtype) || !train_dtype_ok(out_dtype))
    return set_error(MUON_ERR_BAD_DTYPE, "table and out must be fp32 or bf16");
  if (ld_out < dim) return set_error(MUON_ERR_BAD_SHAPE, "ld_out < dim");
  if (n == 0) return MUON_OK;
  if (table == nullptr || ids == nullptr || out == nullptr)
    return set_error(MUON_ERR_INVALID_ARG, "table, ids or out is null");
  const bool tb = table_dtype == MUON_DTYPE_BF16, ob = out_dtype == MUON_DTYPE_BF16;
#define MUON_EMBED_FWD(TT, TO)                                                              \
  (ids_64 ? run_fwd<TT, TO, int64_t>(table, ids, n, vocab, dim, scale, out, ld_out, stream) \
          : run_fwd<TT, TO, int32_t>(table, ids, n, vocab, dim, scale, out, ld_out, stream))
  if (tb && ob) MUON_EMBED_FWD(uint16_t, uint16_t);
  else if (tb) MUON_EMBED_FWD(uint16_t, float);
  else if (ob) MUON_EMBED_FWD(float, uint16_t);
  else MUON_EMBED_FWD(float, float);
#undef MUON_EMBED_FWD
  return check_launch("embedding lookup launch");
}

size_t embed_backward_workspace_size(int64_t n, int64_t vocab, int64_t dim) {
  if (n <= 0 || check_token_sizes(n, vocab, dim) != MUON_OK) return 0;
  return embed_ws(n, dim).total;
}

int embed_backward(const void* dout, int32_t dout_dtype, int64_t ld_dout, const void* ids,
                   int32_t ids_64, int64_t n, float scale, void* dtable, int32_t dtable_dtype,
                   int64_t vocab, int64_t dim, int32_t accumulate, void* workspace,
                   size_t workspace_bytes, hipStream_t stream) {
  const int rc = check_sizes(n, vocab, dim, scale);
  if (rc != MUON_OK) return rc;
  if (!train_dtype_ok(dout_dtype) || !train_dtype_ok(dtable_dtype))
    return set_error(MUON_ERR_BAD_DTYPE, "dout and dtable must be fp32 or bf16");
  if (ld_dout < dim) return set_error(MUON_ERR_BAD_SHAPE, "ld_dout < dim");
  if (dtable == nullptr) return set_error(MUON_ERR_INVALID_ARG, "dtable is null");
  if (n == 0) {
    if (accumulate) return MUON_OK;
  } else if (dout == nullptr || ids == nullptr) {
    return set_error(MUON_ERR_INVALID_ARG, "dout or ids is null");
  }
  const EmbedWs w = embed_ws(n, dim);
  if (n > 0 && (workspace == nullptr || workspace_bytes < w.total ||
                reinterpret_cast<uintptr_t>(workspace) % 256 != 0))
    return set_error(MUON_ERR_WORKSPACE_TOO_SMALL,
                     "embed_backward needs " + std::to_string(w.total) +
                         " bytes of workspace, 256-byte aligned");
  const BackwardArgs a{dout, ids, ld_dout, n, vocab, dim, scale, dtable, accumulate != 0,
                       static_cast<char*>(workspace)};
  const bool db = dout_dtype == MUON_DTYPE_BF16, gb = dtable_dtype == MUON_DTYPE_BF16;
  if (db && gb) run_backward<uint16_t, uint16_t>(a, w, ids_64 != 0, stream);
  else if (db) run_backward<uint16_t, float>(a, w, ids_64 != 0, stream);
  else if (gb) run_backward<float, uint16_t>(a, w, ids_64 != 0, stream);
  else run_backward<float, float>(a, w, ids_64 != 0, stream);
  return check_launch("embedding gradient launch");
}

}  // extern "C"
