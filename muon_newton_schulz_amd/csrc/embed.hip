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
// the sorted list into chunks of kChunk positions and sums each run of
// equal ids inside a chunk in fp32 registers.  A run that lies inside its
// chunk is finished there; a run that crosses a chunk border leaves one
// fp32 partial row per chunk, which a second kernel adds in chunk order.
// A frequent token therefore spreads over as many workgroups as a rare one.
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

template <typename TT, typename TO, typename ID>
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
      store8(out + (t0 + r) * ld + c, x[r]);
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
// LSD radix sort of (key, position) by key, at most kMaxBits bits a pass.
// key = id, or vocab for an id outside [0, vocab), which puts the positions
// without a row last.  Stable: each wave owns a contiguous part of its
// workgroup's keys and places 64 keys at a time, a key's rank among equal
// digits of the 64 being the number of lower lanes that hold the digit.

constexpr int kMaxBits = 9;
constexpr int kMaxBins = 1 << kMaxBits;

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

// Zeroes the table gradient: the part of workgroup `b` of `nb`.
template <typename TG>
__device__ __forceinline__ void zero_part(TG* g, int64_t total, int64_t b, int64_t nb,
                                          int threads) {
  // 16-byte stores on the aligned middle, the ragged ends by workgroup 0
  const int64_t per = 16 / sizeof(TG);
  const int64_t mis = static_cast<int64_t>((reinterpret_cast<uintptr_t>(g) & 15) / sizeof(TG));
  int64_t head = mis ? per - mis : 0;
  if (head > total) head = total;
  const int64_t n16 = (total - head) / per;
  u32x4_t* v = reinterpret_cast<u32x4_t*>(g + head);
  for (int64_t i = b * threads + threadIdx.x; i < n16; i += nb * threads) v[i] = u32x4_t{0, 0, 0, 0};
  if (b == 0) {
    if (static_cast<int64_t>(threadIdx.x) < head) g[threadIdx.x] = TG{};
    const int64_t t = head + n16 * per + threadIdx.x;
    if (t < total) g[t] = TG{};
  }
}

// Up to kSmallN keys: one workgroup sorts them in LDS in one launch, while
// the other workgroups of the launch zero the table gradient.
constexpr int kSmallN = 8192;
constexpr int kSmallThreads = 1024;
constexpr int kSmallWaves = kSmallThreads / 64;

template <typename ID, typename TG>
__global__ __launch_bounds__(kSmallThreads) void k_sort_small(
    const ID* __restrict__ ids, int n, int64_t vocab, int bits, int passes,
    uint32_t* __restrict__ keys_out, uint32_t* __restrict__ pos_out, TG* __restrict__ dtable,
    int64_t total) {
  __shared__ uint32_t key[2][kSmallN];
  __shared__ uint16_t pos[2][kSmallN];
  __shared__ uint32_t cnt[kSmallWaves][kMaxBins];
  __shared__ uint32_t base[kMaxBins], tmp[kSmallWaves];
  if (blockIdx.x > 0) {
    zero_part(dtable, total, blockIdx.x - 1, gridDim.x - 1, kSmallThreads);
    return;
  }
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const uint32_t vocab32 = static_cast<uint32_t>(vocab);
  for (int i = t; i < n; i += kSmallThreads) {
    const int64_t v = static_cast<int64_t>(ids[i]);
    key[0][i] = v >= 0 && v < vocab ? static_cast<uint32_t>(v) : vocab32;
    pos[0][i] = static_cast<uint16_t>(i);
  }
  // contiguous part of each wave, in steps of 64
  const int part = ((n + kSmallWaves - 1) / kSmallWaves + 63) / 64 * 64;
  const int lo = w * part, hi = lo + part < n ? lo + part : n;
  const int bins = 1 << bits;
  const uint32_t mask = static_cast<uint32_t>(bins) - 1u;
  int cur = 0;
  for (int p = 0; p < passes; ++p) {
    const int shift = p * bits;
    for (int i = t; i < kSmallWaves * kMaxBins; i += kSmallThreads) cnt[0][i] = 0;
    __syncthreads();
    for (int i = lo + lane; i < hi; i += 64) atomicAdd(&cnt[w][(key[cur][i] >> shift) & mask], 1u);
    __syncthreads();
    for (int b = t; b < bins; b += kSmallThreads) {
      uint32_t s = 0;
      for (int k = 0; k < kSmallWaves; ++k) {
        const uint32_t c = cnt[k][b];
        cnt[k][b] = s;
        s += c;
      }
      base[b] = s;
    }
    __syncthreads();
    block_exclusive_scan<kSmallThreads>(base, bins, tmp);
    for (int i0 = lo; i0 < hi; i0 += 64) {
      const int i = i0 + lane;
      const bool on = i < hi;
      const uint32_t k = on ? key[cur][i] : 0u;
      const uint32_t d = (k >> shift) & mask;
      const uint64_t m = match_digit(d, bits, __ballot(on));
      if (on) {
        const uint32_t rank = __popcll(m & ((1ull << lane) - 1ull));
        const uint32_t to = base[d] + cnt[w][d] + rank;
        key[cur ^ 1][to] = k;
        pos[cur ^ 1][to] = pos[cur][i];
        // the last lane of the digit moves the wave's counter on
        if ((m >> lane) == 1ull) cnt[w][d] += __popcll(m);
      }
      wave_sync();  // the wave's next 64 keys read the counters just moved
    }
    __syncthreads();
    cur ^= 1;
  }
  for (int i = t; i < n; i += kSmallThreads) {
    keys_out[i] = key[cur][i];
    pos_out[i] = pos[cur][i];
  }
}

// More keys: per pass a histogram per workgroup, a scan over all of them,
// and a stable scatter.
constexpr int kSortThreads = 256;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortKeys = 4096;  // keys per workgroup
constexpr int kWaveKeys = kSortKeys / kSortWaves;

__device__ __forceinline__ uint32_t clip_key(int64_t v, int64_t vocab) {
  return static_cast<uint32_t>(v >= 0 && v < vocab ? v : vocab);
}

// The first pass reads the ids themselves (FIRST); its launch has zero_blocks
// more workgroups, which zero the table gradient.
template <bool FIRST, typename ID, typename TG>
__global__ __launch_bounds__(kSortThreads) void k_sort_hist(
    const ID* __restrict__ ids, const uint32_t* __restrict__ keys, int64_t n, int64_t vocab,
    int shift, int bits, int n_blocks, uint32_t* __restrict__ hist, TG* __restrict__ dtable,
    int64_t total) {
  if (FIRST && static_cast<int>(blockIdx.x) >= n_blocks) {
    zero_part(dtable, total, blockIdx.x - n_blocks, gridDim.x - n_blocks, kSortThreads);
    return;
  }
  __shared__ uint32_t cnt[kMaxBins];
  const int bins = 1 << bits;
  for (int b = threadIdx.x; b < bins; b += kSortThreads) cnt[b] = 0;
  __syncthreads();
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kSortKeys;
  for (int k = threadIdx.x; k < kSortKeys; k += kSortThreads)
    if (i0 + k < n) {
      const uint32_t key = FIRST ? clip_key(static_cast<int64_t>(ids[i0 + k]), vocab) : keys[i0 + k];
      atomicAdd(&cnt[(key >> shift) & (bins - 1)], 1u);
    }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads)
    hist[static_cast<int64_t>(b) * n_blocks + blockIdx.x] = cnt[b];
}

// exclusive scan of m entries in place, one workgroup
__global__ __launch_bounds__(1024) void k_sort_scan(uint32_t* __restrict__ h, int64_t m) {
  __shared__ uint32_t tmp[16];
  __shared__ uint32_t carry_s;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  uint32_t carry = 0;
  for (int64_t i0 = 0; i0 < m; i0 += 4096) {
    const int64_t i = i0 + 4 * t;
    uint32_t v[4], s = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = i + k < m ? h[i + k] : 0;
      s += v[k];
    }
    uint32_t sc = s;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t u = __shfl_up(sc, o, 64);
      if (lane >= o) sc += u;
    }
    if (lane == 63) tmp[w] = sc;
    __syncthreads();
    uint32_t base = carry;
    for (int k = 0; k < w; ++k) base += tmp[k];
    uint32_t ex = base + sc - s;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i + k < m) h[i + k] = ex;
      ex += v[k];
    }
    if (t == 1023) carry_s = base + sc;
    __syncthreads();
    carry = carry_s;
  }
}

template <bool FIRST, typename ID>
__global__ __launch_bounds__(kSortThreads) void k_sort_scatter(
    const ID* __restrict__ ids, const uint32_t* __restrict__ keys,
    const uint32_t* __restrict__ pos, int64_t n, int64_t vocab, int shift, int bits, int n_blocks,
    const uint32_t* __restrict__ hist, uint32_t* __restrict__ keys_out,
    uint32_t* __restrict__ pos_out) {
  __shared__ uint32_t cnt[kSortWaves][kMaxBins];
  const int bins = 1 << bits;
  const uint32_t mask = static_cast<uint32_t>(bins) - 1u;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  for (int i = t; i < kSortWaves * kMaxBins; i += kSortThreads) cnt[0][i] = 0;
  __syncthreads();
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * kSortKeys + w * kWaveKeys;
  uint32_t k[kWaveKeys / 64];
#pragma unroll
  for (int r = 0; r < kWaveKeys / 64; ++r) {
    const int64_t i = lo + r * 64 + lane;
    k[r] = 0;
    if (i < n) {
      k[r] = FIRST ? clip_key(static_cast<int64_t>(ids[i]), vocab) : keys[i];
      atomicAdd(&cnt[w][(k[r] >> shift) & mask], 1u);
    }
  }
  __syncthreads();
  for (int b = t; b < bins; b += kSortThreads) {
    uint32_t s = hist[static_cast<int64_t>(b) * n_blocks + blockIdx.x];
    for (int j = 0; j < kSortWaves; ++j) {
      const uint32_t c = cnt[j][b];
      cnt[j][b] = s;
      s += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kWaveKeys / 64; ++r) {
    const int64_t i = lo + r * 64 + lane;
    const bool on = i < n;
    const uint32_t d = (k[r] >> shift) & mask;
    const uint64_t m = match_digit(d, bits, __ballot(on));
    if (on) {
      const uint32_t to = cnt[w][d] + __popcll(m & ((1ull << lane) - 1ull));
      keys_out[to] = k[r];
      pos_out[to] = FIRST ? static_cast<uint32_t>(i) : pos[i];
      if ((m >> lane) == 1ull) cnt[w][d] += __popcll(m);
    }
    wave_sync();
  }
}

// -------------------------------------------------------------------- sums

constexpr int kChunk = 32;

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

template <typename TD, typename TG>
__global__ __launch_bounds__(kThreads) void k_embed_runs(
    const TD* __restrict__ dout, int64_t ld, const uint32_t* __restrict__ keys,
    const uint32_t* __restrict__ pos, int64_t n, int64_t vocab, int64_t dim, int64_t dim_p,
    float scale, int accumulate, TG* __restrict__ dtable, float* __restrict__ parts) {
  const int64_t chunk = blockIdx.x;
  const int64_t s0 = chunk * kChunk;
  const int len = static_cast<int>(n - s0 < kChunk ? n - s0 : kChunk);
  const int64_t c = static_cast<int64_t>(blockIdx.y) * kCols + threadIdx.x * 8;
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
__global__ __launch_bounds__(kThreads) void k_embed_join(
    const uint32_t* __restrict__ keys, int64_t n, int64_t n_chunks, int64_t vocab, int64_t dim,
    int64_t dim_p, float scale, int accumulate, TG* __restrict__ dtable, float* parts) {
  const int64_t chunk = blockIdx.x;
  const int64_t end = (chunk + 1) * kChunk;
  if (end >= n) return;
  const uint32_t key = keys[end - 1];
  if (key == static_cast<uint32_t>(vocab) || keys[end] != key) return;
  // the run started in an earlier chunk: that chunk joins it
  if (chunk > 0 && keys[end - kChunk] == key && keys[end - kChunk - 1] == key) return;
  const int64_t c = static_cast<int64_t>(blockIdx.y) * kCols + threadIdx.x * 8;
  if (c >= dim) return;
  // the last chunk that the run reaches: first position whose key exceeds it
  int64_t lo = end, hi = n;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (keys[mid] <= key) lo = mid + 1;
    else hi = mid;
  }
  const int64_t last = (lo - 1) / kChunk;
  float acc[8];
  load8(partial_row(parts, chunk, 1, dim_p) + c, acc);
  int64_t k = chunk + 1;
  for (; k + 3 <= last; k += 4) {
    float x[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u) load8(partial_row(parts, k + u, 0, dim_p) + c, x[u]);
#pragma unroll
    for (int u = 0; u < 4; ++u)
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

// -------------------------------------------------------------------- host

int key_bits(int64_t vocab) {
  int b = 1;
  while ((static_cast<int64_t>(1) << b) <= vocab) ++b;  // the largest key is vocab
  return b;
}

struct EmbedWs {
  size_t keys[2], pos[2], hist, parts, total;
  int64_t blocks, chunks, dim_p;
};
EmbedWs embed_ws(int64_t n, int64_t dim) {
  EmbedWs w{};
  w.blocks = (n + kSortKeys - 1) / kSortKeys;
  w.chunks = (n + kChunk - 1) / kChunk;
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

template <typename TT, typename TO, typename ID>
void run_fwd(const void* table, const void* ids, int64_t n, int64_t vocab, int64_t dim,
             float scale, void* out, int64_t ld, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((n + kRows - 1) / kRows),
                  static_cast<unsigned>((dim + kCols - 1) / kCols));
  hipLaunchKernelGGL((k_embed_fwd<TT, TO, ID>), grid, dim3(kThreads), 0, s,
                     static_cast<const TT*>(table), static_cast<const ID*>(ids), n, vocab, dim,
                     scale, static_cast<TO*>(out), ld);
}

// workgroups that zero the table gradient beside the sort: enough to reach
// the write rate, few enough that each has several stores
int zero_blocks(int64_t total, size_t size, int threads) {
  const int64_t pieces = (total * static_cast<int64_t>(size) + 16 * threads * 4 - 1) / (16 * threads * 4);
  return static_cast<int>(pieces < 4096 ? (pieces < 1 ? 1 : pieces) : 4096);
}

template <typename ID, typename TG>
void run_sort(const void* ids_v, int64_t n, int64_t vocab, const EmbedWs& w, char* ws,
              void* dtable, int64_t total, bool zero, hipStream_t s, int* cur_out) {
  const ID* ids = static_cast<const ID*>(ids_v);
  uint32_t* keys[2] = {reinterpret_cast<uint32_t*>(ws + w.keys[0]),
                       reinterpret_cast<uint32_t*>(ws + w.keys[1])};
  uint32_t* pos[2] = {reinterpret_cast<uint32_t*>(ws + w.pos[0]),
                      reinterpret_cast<uint32_t*>(ws + w.pos[1])};
  uint32_t* hist = reinterpret_cast<uint32_t*>(ws + w.hist);
  const int all = key_bits(vocab);
  const int passes = (all + kMaxBits - 1) / kMaxBits;
  const int bits = (all + passes - 1) / passes;
  TG* dt = static_cast<TG*>(dtable);
  if (n <= kSmallN) {
    const int zb = zero ? zero_blocks(total, sizeof(TG), kSmallThreads) : 0;
    hipLaunchKernelGGL((k_sort_small<ID, TG>), dim3(1 + zb), dim3(kSmallThreads), 0, s, ids,
                       static_cast<int>(n), vocab, bits, passes, keys[0], pos[0], dt, total);
    *cur_out = 0;
    return;
  }
  const int nb = static_cast<int>(w.blocks);
  int cur = 0;
  for (int p = 0; p < passes; ++p) {
    const int shift = p * bits;
    if (p == 0) {
      const int zb = zero ? zero_blocks(total, sizeof(TG), kSortThreads) : 0;
      hipLaunchKernelGGL((k_sort_hist<true, ID, TG>), dim3(nb + zb), dim3(kSortThreads), 0, s,
                         ids, nullptr, n, vocab, shift, bits, nb, hist, dt, total);
    } else {
      hipLaunchKernelGGL((k_sort_hist<false, ID, TG>), dim3(nb), dim3(kSortThreads), 0, s, ids,
                         keys[cur], n, vocab, shift, bits, nb, hist, dt, total);
    }
    hipLaunchKernelGGL(k_sort_scan, dim3(1), dim3(1024), 0, s, hist,
                       static_cast<int64_t>(nb) << bits);
    if (p == 0)
      hipLaunchKernelGGL((k_sort_scatter<true, ID>), dim3(nb), dim3(kSortThreads), 0, s, ids,
                         nullptr, nullptr, n, vocab, shift, bits, nb, hist, keys[cur ^ 1],
                         pos[cur ^ 1]);
    else
      hipLaunchKernelGGL((k_sort_scatter<false, ID>), dim3(nb), dim3(kSortThreads), 0, s, ids,
                         keys[cur], pos[cur], n, vocab, shift, bits, nb, hist, keys[cur ^ 1],
                         pos[cur ^ 1]);
    cur ^= 1;
  }
  *cur_out = cur;
}

template <typename TG>
void run_sums(const void* dout, int32_t dout_dtype, int64_t ld, const uint32_t* keys,
              const uint32_t* pos, int64_t n, int64_t vocab, int64_t dim, const EmbedWs& w,
              float scale, int accumulate, void* dtable, float* parts, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(w.chunks),
                  static_cast<unsigned>((dim + kCols - 1) / kCols));
  TG* dt = static_cast<TG*>(dtable);
  if (dout_dtype == MUON_DTYPE_BF16)
    hipLaunchKernelGGL((k_embed_runs<uint16_t, TG>), grid, dim3(kThreads), 0, s,
                       static_cast<const uint16_t*>(dout), ld, keys, pos, n, vocab, dim, w.dim_p,
                       scale, accumulate, dt, parts);
  else
    hipLaunchKernelGGL((k_embed_runs<float, TG>), grid, dim3(kThreads), 0, s,
                       static_cast<const float*>(dout), ld, keys, pos, n, vocab, dim, w.dim_p,
                       scale, accumulate, dt, parts);
  if (w.chunks > 1)
    hipLaunchKernelGGL(k_embed_join<TG>, grid, dim3(kThreads), 0, s, keys, n, w.chunks, vocab,
                       dim, w.dim_p, scale, accumulate, dt, parts);
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
  char* ws = static_cast<char*>(workspace);
  const int64_t total = vocab * dim;
  const bool gb = dtable_dtype == MUON_DTYPE_BF16;
  int cur = 0;
  const bool zero = accumulate == 0;
  if (ids_64) {
    if (gb) run_sort<int64_t, uint16_t>(ids, n, vocab, w, ws, dtable, total, zero, stream, &cur);
    else run_sort<int64_t, float>(ids, n, vocab, w, ws, dtable, total, zero, stream, &cur);
  } else {
    if (gb) run_sort<int32_t, uint16_t>(ids, n, vocab, w, ws, dtable, total, zero, stream, &cur);
    else run_sort<int32_t, float>(ids, n, vocab, w, ws, dtable, total, zero, stream, &cur);
  }
  if (n > 0) {
    const uint32_t* keys = reinterpret_cast<const uint32_t*>(ws + w.keys[cur]);
    const uint32_t* pos = reinterpret_cast<const uint32_t*>(ws + w.pos[cur]);
    float* parts = reinterpret_cast<float*>(ws + w.parts);
    if (gb) run_sums<uint16_t>(dout, dout_dtype, ld_dout, keys, pos, n, vocab, dim, w, scale,
                               accumulate, dtable, parts, stream);
    else run_sums<float>(dout, dout_dtype, ld_dout, keys, pos, n, vocab, dim, w, scale,
                         accumulate, dtable, parts, stream);
  }
  return check_launch("embedding gradient launch");
}

}  // extern "C"
