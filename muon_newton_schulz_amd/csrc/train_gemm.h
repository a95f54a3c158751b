// Tile cores of the matrix products behind the vocabulary loss
// (lm_loss.hip) and the expert products (experts.hip).
//
// A core computes one output tile C[i][j] = sum_k P(i, k) Q(j, k), i < BM,
// j < BN, with four waves in a WM x WN grid, each MI x NJ blocks of 32x32
// on the matrix cores with fp32 accumulation.  An operand is K-contiguous
// (element (r, k) at p[r * ld + k]) or K-strided (at p[k * ld + r]); pn and
// qn are the rows of P and Q that exist from the tile's first row on (the
// others count as zero and are not read), K the length of the sum.  run<true>
// adds to what acc holds; a second run may follow a first at once.
//
// Accumulators (A operand = Q, B operand = P): acc[bj][bi][4 q + e] of a
// lane is element
//   i = wi * 32 MI + 32 bi + lane % 32,
//   j = wj * 32 NJ + 32 bj + 8 q + 4 (lane / 32) + e,
// so a lane holds four consecutive columns of one row.
#pragma once

#include <cmath>
#include <type_traits>

#include "train_common.h"

namespace muon {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

template <int NJ, int MI>
__device__ __forceinline__ void zero_acc(f32x16_t (&acc)[NJ][MI]) {
#pragma unroll
  for (int a = 0; a < NJ; ++a)
#pragma unroll
    for (int b = 0; b < MI; ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[a][b][v] = 0.0f;
}

template <int NJ, int MI>
__device__ __forceinline__ void scale_acc(f32x16_t (&acc)[NJ][MI], float c) {
#pragma unroll
  for (int a = 0; a < NJ; ++a)
#pragma unroll
    for (int b = 0; b < MI; ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[a][b][v] *= c;
}

// Calls f(i, j, value) for every group of four columns of this thread.
template <typename Core, typename F>
__device__ __forceinline__ void each_quad(f32x16_t (&acc)[Core::NJ][Core::MI], F&& f) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i0 = (wave % Core::WM) * 32 * Core::MI + (lane & 31);
  const int j0 = (wave / Core::WM) * 32 * Core::NJ + 4 * (lane >> 5);
#pragma unroll
  for (int bj = 0; bj < Core::NJ; ++bj)
#pragma unroll
    for (int bi = 0; bi < Core::MI; ++bi)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4_t v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[bj][bi][4 * q + e];
        f(i0 + 32 * bi, j0 + 32 * bj + 8 * q, v);
      }
}

// Four consecutive columns of a row, `left` >= 1 of which exist.
template <typename TO>
__device__ __forceinline__ void store_quad(TO* p, int left, f32x4_t v) {
  if (left >= 4) {
    if constexpr (sizeof(TO) == 4) {
      __builtin_memcpy(p, &v, 16);
    } else {
      const u32x2_t w = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
      __builtin_memcpy(p, &w, 8);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < left) from_f32(v[e], p + e);
  }
}

// C[i][j] = acc (+ add[i][j]) for i < rows, j < cols, no alignment needed.
// add may be C.  (Its stores are parts of lines, which the caches have to put
// together: with nontemporal ones the weight gradient of 700 x 1281 x 1021,
// 20 experts, took 136 us instead of 27.)
template <typename Core, typename TO, typename TA>
__device__ __forceinline__ void write_quads(f32x16_t (&acc)[Core::NJ][Core::MI], TO* C, int64_t ldc,
                                            const TA* add, int64_t lda, int rows, int cols) {
  each_quad<Core>(acc, [&](int i, int j, f32x4_t v) {
    if (i >= rows || j >= cols) return;
    if (add != nullptr) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j + e < cols) v[e] += to_f32(add[i * lda + j + e]);
    }
    store_quad(C + i * ldc + j, cols - j, v);
  });
}

// Tile t of an nx x ny grid of tiles: bands of kBand row tiles, column by
// column.  Workgroups go to the 8 XCDs in turn, so workgroup b works in the
// (b % 8)-th eighth of this list: the 32 CUs of an XCD run neighbouring
// tiles and share operands in their L2.
constexpr int kXcds = 8, kBand = 8;
__device__ __forceinline__ void tile_at(int64_t t, int64_t nx, int64_t ny, int& x, int& y) {
  const int64_t band = t / (kBand * ny), r = t - band * kBand * ny;
  const int64_t h = nx - band * kBand < kBand ? nx - band * kBand : kBand;
  x = static_cast<int>(band * kBand + r % h);
  y = static_cast<int>(r / h);
}

// Waits for this wave's LDS accesses and then for the workgroup.  Unlike
// __syncthreads it leaves vector memory instructions (DMA, stores) in
// flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// One tile's operands; K <= 0 gives zeros.
template <typename T>
struct TileArgs {
  const T *P, *Q;
  int64_t ldp, ldq;
  int pn, qn, K;
};

// The tile of this workgroup among nx x ny (tile_at), if it has one.  A launch
// of tile_blocks(nx, ny) workgroups covers them all.
__device__ __forceinline__ bool my_tile(int64_t nx, int64_t ny, int& x, int& y) {
  const int64_t total = nx * ny, per = (total + kXcds - 1) / kXcds;
  const int64_t k = blockIdx.x / kXcds, t = blockIdx.x % kXcds * per + k;
  if (k >= per || t >= total) return false;
  tile_at(t, nx, ny, x, y);
  return true;
}
inline unsigned tile_blocks(int64_t nx, int64_t ny) {
  return static_cast<unsigned>((nx * ny + kXcds - 1) / kXcds * kXcds);
}
// Whether a launch holds that many: fewer than 2^32 threads.
inline bool tiles_fit(int64_t nx, int64_t ny) { return nx * ny <= (int64_t{1} << 24) - kXcds; }

// 8 k (bf16) or 4 k (fp32) of a 16-wide (8-wide) k step from LDS:
// transposed read of a K-strided tile.  Within each group of 16 lanes, lane
// l receives element l % 4 of the 8-byte blocks addressed by lanes
// 4 q + l / 4, q = 0..3.
__device__ __forceinline__ s16x4_t lds_read_tr(const uint16_t* p) {
  typedef __attribute__((address_space(3))) s16x4_t* lds_t;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)(p));
}

// 16 bytes of an operand tile of B rows (columns) by CK k: piece pc counts
// along the memory's rows.  What lies past row n or k = K is zero.
template <typename T, bool KS, int B, int CK>
__device__ __forceinline__ u32x4_t load_piece(const T* p, int64_t ld, int n, int K, int k0, int pc) {
  constexpr int E = 16 / sizeof(T);
  constexpr int PR = (KS ? B : CK) / E;  // pieces to a row
  const int row = pc / PR, col = pc % PR * E;
  const int r = KS ? col : row, k = k0 + (KS ? row : col);
  const int left = KS ? (k < K ? n - r : 0) : (r < n ? K - k : 0);
  const T* a = p + static_cast<int64_t>(KS ? k : r) * ld + (KS ? r : k);
  u32x4_t w = {0, 0, 0, 0};
  if (left >= E) {
    __builtin_memcpy(&w, a, 16);
  } else if (left > 0) {
    T x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = e < left ? a[e] : T{};
    __builtin_memcpy(&w, x, 16);
  }
  return w;
}

// ------------------------------------------------------------ any operands
//
// The core for operands off the 16-byte grid, and for fp32: 128x128 or 64x64
// tiles, 64 bytes of k at a time (32 bf16, 16 fp32) through registers into
// double-buffered LDS, the next step's loads in flight during the current
// step's matrix instructions.  Loads need no alignment; a piece of 16 bytes
// that crosses the end of a row (or of the tile's columns) is read element
// by element, so nothing outside the operands is touched.
// fp32 runs on v_mfma_f32_32x32x2_f32: lane l of instruction s of a group
// of 8 k supplies k = 4 (l / 32) + s, for both operands.  Its sums restart
// every kFlush steps (256 k) and are added up beside them, so that rounding
// grows with the square root of 256 and of K / 256 instead of that of K.
template <typename T, bool PKS, bool QKS, int B>
struct AnyCore {
  static constexpr int BM = B, BN = B, MI = B / 64, NJ = B / 64, WM = 2, WN = 2;
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr int E = 16 / sizeof(T);   // elements per 16-byte piece
  static constexpr int CK = 4 * E;           // k per step
  static constexpr int H = B / 64;           // pieces of an operand per thread
  // LDS strides in elements.  K-contiguous rows of 64 bytes are padded to
  // 80, so that 16-byte reads of consecutive rows spread over the banks;
  // K-strided rows of B columns by 8 elements, so that the k rows the two
  // lane halves read differ by half the banks.
  static constexpr int SC = CK + E, SS = B + 8;
  static constexpr int kOperandBytes =
      (B * SC > CK * SS ? B * SC : CK * SS) * static_cast<int>(sizeof(T));
  static constexpr int kLdsBytes = 4 * kOperandBytes;
  static constexpr int kWaves = B == 128 ? 2 : 4;  // per SIMD, at least
  static constexpr bool kGrid = false;
  static constexpr int kFlush = 16;
  static __device__ __forceinline__ char* lds() {
    __shared__ __attribute__((aligned(16))) char mem[kLdsBytes];
    return mem;
  }

  template <bool KS>
  static __device__ __forceinline__ T* lds_piece(T* s, int pc) {
    constexpr int PR = B / E;
    return KS ? s + (pc / PR) * SS + (pc % PR) * E : s + (pc >> 2) * SC + (pc & 3) * E;
  }
  // operand fragment of 32-row block at row b, k step g (16 bf16, 8 fp32)
  template <bool KS>
  static __device__ __forceinline__ auto frag(const T* s, int b, int g, int lane) {
    if constexpr (F32) {
      f32x4_t f;
      const int k = 8 * g + 4 * (lane >> 5), r = b + (lane & 31);
      if constexpr (KS) {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = s[(k + e) * SS + r];
      } else {
        f = *reinterpret_cast<const f32x4_t*>(s + r * SC + k);
      }
      return f;
    } else {
      const int k = 16 * g + 8 * (lane >> 5);
      if constexpr (KS) {
        const int l = lane & 15;
        const uint16_t* a = s + (k + (l >> 2)) * SS + b + 16 * ((lane >> 4) & 1) + 4 * (l & 3);
        const s16x4_t lo = lds_read_tr(a), hi = lds_read_tr(a + 4 * SS);
        return __builtin_bit_cast(bf16x8_t,
                                  __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      } else {
        return *reinterpret_cast<const bf16x8_t*>(s + (b + (lane & 31)) * SC + k);
      }
    }
  }

  template <bool ADD = false>
  static __device__ __forceinline__ void run(const TileArgs<T>& w, f32x16_t (&acc)[NJ][MI]) {
    run_in<ADD>(w, acc, lds());
  }
  template <bool ADD = false>
  static __device__ __forceinline__ void run_in(const TileArgs<T>& w, f32x16_t (&acc)[NJ][MI],
                                                char* smem) {
    const T *P = w.P, *Q = w.Q;
    const int64_t ldp = w.ldp, ldq = w.ldq;
    const int pn = w.pn, qn = w.qn, K = w.K;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int wi = wave % WM, wj = wave / WM;
    u32x4_t pr[H], qr[H];
    auto load = [&](int k0) {
#pragma unroll
      for (int h = 0; h < H; ++h) {
        pr[h] = load_piece<T, PKS, B, CK>(P, ldp, pn, K, k0, t + 256 * h);
        qr[h] = load_piece<T, QKS, B, CK>(Q, ldq, qn, K, k0, t + 256 * h);
      }
    };
    auto buf = [&](int b, int op) {
      return reinterpret_cast<T*>(smem + (2 * b + op) * kOperandBytes);
    };
    auto store = [&](int b) {
#pragma unroll
      for (int h = 0; h < H; ++h) {
        *reinterpret_cast<u32x4_t*>(lds_piece<PKS>(buf(b, 0), t + 256 * h)) = pr[h];
        *reinterpret_cast<u32x4_t*>(lds_piece<QKS>(buf(b, 1), t + 256 * h)) = qr[h];
      }
    };
    if constexpr (!ADD) zero_acc(acc);
    if (K <= 0) return;
    const int steps = (K + CK - 1) / CK;
    load(0);
    store(0);  // (no wave reads the buffers of a run before this one any more)
    __syncthreads();
    auto span = [&](f32x16_t (&d)[NJ][MI], int c0, int c1) {
      for (int c = c0; c < c1; ++c) {
        const int b = c & 1;
        if (c + 1 < steps) load((c + 1) * CK);
        const T* ps = buf(b, 0);
        const T* qs = buf(b, 1);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          decltype(frag<PKS>(ps, 0, 0, 0)) p[MI];
          decltype(frag<QKS>(qs, 0, 0, 0)) q[NJ];
#pragma unroll
          for (int i = 0; i < MI; ++i) p[i] = frag<PKS>(ps, wi * 32 * MI + 32 * i, g, lane);
#pragma unroll
          for (int j = 0; j < NJ; ++j) q[j] = frag<QKS>(qs, wj * 32 * NJ + 32 * j, g, lane);
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int i = 0; i < MI; ++i) {
              if constexpr (F32) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  d[j][i] = __builtin_amdgcn_mfma_f32_32x32x2f32(q[j][e], p[i][e], d[j][i], 0, 0, 0);
              } else {
                d[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(q[j], p[i], d[j][i], 0, 0, 0);
              }
            }
        }
        if (c + 1 < steps) store(b ^ 1);
        __syncthreads();
      }
    };
    if constexpr (F32) {
      for (int c0 = 0; c0 < steps; c0 += kFlush) {
        f32x16_t part[NJ][MI];
        zero_acc(part);
        span(part, c0, min(c0 + kFlush, steps));
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < MI; ++i) acc[j][i] += part[j][i];
      }
    } else {
      span(acc, 0, steps);
    }
  }

  template <bool STREAM = false, typename TO, typename TA>
  static __device__ __forceinline__ void write(f32x16_t (&acc)[NJ][MI], TO* C, int64_t ldc,
                                               const TA* add, int64_t lda, int rows, int cols) {
    write_quads<AnyCore>(acc, C, ldc, add, lda, rows, cols);
  }
};

// ------------------------------------------------------- fp32 in three bf16
//
// fp32 products on the bf16 matrix cores: an operand x is the sum of three
// bf16 values, hi = bf16(x), mid = bf16(x - hi), lo = bf16(x - hi - mid),
// exactly while lo is in fp32's normal range or 0, and of the nine products
// the six above 2^-26 of the largest are added, smallest first, in fp32
// (products of bf16 are exact in fp32).  The result is as accurate as a sum of
// fp32 products (Henry, Tang, Heinecke, "Leveraging the bfloat16 artificial
// intelligence datatype for higher-precision computations", 2019).  Six bf16
// instructions take 192 cycles for 16 k, the fp32 ones 512.
// An operand that is not finite, or rounds to an infinite hi, makes its
// results NaN here, and one below 2^-109 loses bits of its lo and mid under
// bf16's smallest value, 2^-133 (a third of the mantissa at 2^-120); its lo is
// below fp32's normal range (which starts for some values at 2^-103).  A tile
// with either is computed again on the fp32 instructions; results that are not
// finite, and those of rows and columns with such a small operand, are taken
// from there.  Looking for small ones is one instruction a value: 16384 rows of
// 8 experts, 2048 x 2048, 807 us with it and 778 without (by the bits of x, for
// 0 < |x| < 2^-107: 833), loss 515 x 33001 x 500 backward 452 and 439.  With one
// in every tile, small or not finite, a product takes 3.2 times as long.
// 32 k a step; the operands are split on their way into LDS (single buffer;
// two to four workgroups share a CU).  Sums restart every 256 k.
template <bool PKS, bool QKS, int B>
struct SplitCore {
  using Exact = AnyCore<float, PKS, QKS, B>;
  using Half = AnyCore<uint16_t, PKS, QKS, B>;  // its fragments and strides
  static constexpr int BM = B, BN = B, MI = B / 64, NJ = B / 64, WM = 2, WN = 2, CK = 32;
  static constexpr int H = B / 32;              // pieces of an operand per thread
  static constexpr int kPlane = Half::kOperandBytes;
  static constexpr int kLdsBytes = 6 * kPlane > Exact::kLdsBytes ? 6 * kPlane : Exact::kLdsBytes;
  static constexpr int kWaves = B == 128 ? 2 : 4;
  static constexpr bool kGrid = false;
  static constexpr int kFlush = 8;
  static __device__ __forceinline__ char* lds() {
    __shared__ __attribute__((aligned(16))) char mem[kLdsBytes];
    return mem;
  }
  // plane k (hi, mid, lo) of operand op
  static __device__ __forceinline__ uint16_t* plane(int op, int k) {
    return reinterpret_cast<uint16_t*>(lds() + (3 * op + k) * kPlane);
  }
  // 0 < |x| < 2^-126
  static __device__ __forceinline__ bool subnormal(float x) {
    return __builtin_amdgcn_classf(x, 0x90);
  }
  // low: set if a lo is of a value below fp32's normal range
  template <bool KS>
  static __device__ __forceinline__ void split_store(int op, int pc, u32x4_t w, bool& low) {
    constexpr int PR = (KS ? B : CK) / 4;
    const int o = pc / PR * (KS ? Half::SS : Half::SC) + pc % PR * 4;
    const f32x4_t x = __builtin_bit_cast(f32x4_t, w);
    f32x2_t a = {x[0], x[1]}, b = {x[2], x[3]};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const u32x2_t h = {pack_bf16(a[0], a[1]), pack_bf16(b[0], b[1])};
      *reinterpret_cast<u32x2_t*>(plane(op, k) + o) = h;
      if (k == 2) break;
      a[0] -= __uint_as_float(h[0] << 16);
      a[1] -= __uint_as_float(h[0] & 0xffff0000u);
      b[0] -= __uint_as_float(h[1] << 16);
      b[1] -= __uint_as_float(h[1] & 0xffff0000u);
    }
    low |= subnormal(a[0]) | subnormal(a[1]) | subnormal(b[0]) | subnormal(b[1]);
  }

  // Marks the rows of an operand that hold a small value, a bit each.
  template <bool KS>
  static __device__ __forceinline__ void mark_small(const float* p, int64_t ld, int n, int K,
                                                    uint32_t* marks) {
    constexpr int PR = (KS ? B : CK) / 4;
    for (int k0 = 0; k0 < K; k0 += CK)
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int pc = threadIdx.x + 256 * h;
        const u32x4_t w = load_piece<float, KS, B, CK>(p, ld, n, K, k0, pc);
        const f32x4_t x = __builtin_bit_cast(f32x4_t, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float a = x[e];
          a -= __uint_as_float(pack_bf16(a, a) << 16);
          a -= __uint_as_float(pack_bf16(a, a) << 16);
          const int r = KS ? pc % PR * 4 + e : pc / PR;
          if (subnormal(a)) atomicOr(&marks[r >> 5], 1u << (r & 31));
        }
      }
  }

  static __device__ __forceinline__ void run(const TileArgs<float>& w, f32x16_t (&acc)[NJ][MI]) {
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int wi = wave % WM, wj = wave / WM;
    bool low = false;
    zero_acc(acc);
    if (w.K <= 0) return;
    u32x4_t pr[H], qr[H];
    auto load = [&](int k0) {
#pragma unroll
      for (int h = 0; h < H; ++h) {
        pr[h] = load_piece<float, PKS, B, CK>(w.P, w.ldp, w.pn, w.K, k0, t + 256 * h);
        qr[h] = load_piece<float, QKS, B, CK>(w.Q, w.ldq, w.qn, w.K, k0, t + 256 * h);
      }
    };
    const int steps = (w.K + CK - 1) / CK;
    load(0);
    for (int c0 = 0; c0 < steps; c0 += kFlush) {
      f32x16_t part[NJ][MI];
      zero_acc(part);
      for (int c = c0; c < min(c0 + kFlush, steps); ++c) {
        __syncthreads();  // the step before is read
#pragma unroll
        for (int h = 0; h < H; ++h) {
          split_store<PKS>(0, t + 256 * h, pr[h], low);
          split_store<QKS>(1, t + 256 * h, qr[h], low);
        }
        __syncthreads();
        if (c + 1 < steps) load((c + 1) * CK);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          bf16x8_t p[3][MI], q[3][NJ];
#pragma unroll
          for (int k = 0; k < 3; ++k) {
#pragma unroll
            for (int i = 0; i < MI; ++i)
              p[k][i] = Half::template frag<PKS>(plane(0, k), wi * 32 * MI + 32 * i, g, lane);
#pragma unroll
            for (int j = 0; j < NJ; ++j)
              q[k][j] = Half::template frag<QKS>(plane(1, k), wj * 32 * NJ + 32 * j, g, lane);
          }
          // (p, q): lo hi, mid mid, hi lo, mid hi, hi mid, hi hi
          constexpr int PK[6] = {2, 1, 0, 1, 0, 0}, QK[6] = {0, 1, 2, 0, 1, 0};
#pragma unroll
          for (int m = 0; m < 6; ++m)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
              for (int i = 0; i < MI; ++i)
                part[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(q[QK[m]][j], p[PK[m]][i],
                                                                     part[j][i], 0, 0, 0);
        }
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[j][i] += part[j][i];
    }
    bool odd = low;  // x - x is 0 unless x is not finite
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) odd |= !(acc[j][i][v] - acc[j][i][v] == 0.0f);
    if (__syncthreads_or(odd)) {
      // only those results are replaced: a row's result does not depend on
      // what the rows beside it hold
      __shared__ uint32_t marks[2][B / 32];
      if (t < 2 * (B / 32)) marks[0][t] = 0u;
      __syncthreads();
      mark_small<PKS>(w.P, w.ldp, w.pn, w.K, marks[0]);
      mark_small<QKS>(w.Q, w.ldq, w.qn, w.K, marks[1]);
      f32x16_t again[NJ][MI];
      Exact::run_in(w, again, lds());  // (its barriers stand between marks and their readers)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          // bit 8 q + e: column 8 q + 4 (lane / 32) + e of the block
          const uint32_t cols = marks[1][wj * NJ + j] >> 4 * (lane >> 5);
          const bool row = (marks[0][wi * MI + i] >> (lane & 31)) & 1u;
#pragma unroll
          for (int v = 0; v < 16; ++v)
            if (row || ((cols >> (8 * (v >> 2) + (v & 3))) & 1u) ||
                !(acc[j][i][v] - acc[j][i][v] == 0.0f))
              acc[j][i][v] = again[j][i][v];
        }
    }
  }

  template <bool STREAM = false, typename TO, typename TA>
  static __device__ __forceinline__ void write(f32x16_t (&acc)[NJ][MI], TO* C, int64_t ldc,
                                               const TA* add, int64_t lda, int rows, int cols) {
    write_quads<SplitCore>(acc, C, ldc, add, lda, rows, cols);
  }
};

// ------------------------------------------------------- aligned bf16 tiles
//
// The core for bf16 operands on the 16-byte grid (base, row stride and row
// length multiples of 8 elements): operand tiles go from memory to LDS by
// DMA (global_load_lds, 16 bytes a lane, no registers), through NS slots of
// BK k each, NS - 1 stages in flight.
//   K-contiguous tile [R rows][BK]: 16-byte chunk c of row r at position
//     c ^ ((r >> 1) & 7) (BK = 64) or c ^ ((r >> 2) & 3) (BK = 32), so that
//     16 consecutive rows' 16-byte reads cover the 64 banks once;
//   K-strided tile [BK][R columns]: 32-column block q of row k at
//     q ^ (k & 3) (R >= 128) or q ^ ((k >> 1) & 1) (R = 64), the same for
//     the transposed reads of four k rows.
// Rows of P and Q past pn, qn are read from the last row there is (their
// results are not used); k past K come from a page of zeros.  Where K is not
// a multiple of 8, a K-contiguous operand's rows hold zeros up to the next.
//
// Each slot is a __shared__ array of its own: the compiler tracks the DMA
// into each separately, and its waits before LDS reads let the newer stages
// stay in flight.

// 16 bytes per lane, memory -> LDS; lane l's data lands at lds + 16 l.  The
// source is a wave-uniform base plus a 32-bit lane offset.
__device__ __forceinline__ void dma16(const char* base, uint32_t voff, char* lds) {
  typedef __attribute__((address_space(1))) void* gbl_t;
  typedef __attribute__((address_space(3))) void* lds_t;
  // one scalar: the address is matched as SGPR base + VGPR offset
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const uint64_t sbase =
      static_cast<uint64_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b >> 32))) << 32 |
      static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b)));
  __builtin_amdgcn_global_load_lds((gbl_t)(reinterpret_cast<const char*>(sbase) + voff),
                                   (lds_t)lds, 16, 0, 0);
}
// the same from an address per lane
__device__ __forceinline__ void dma16_at(const char* p, char* lds) {
  typedef __attribute__((address_space(1))) void* gbl_t;
  typedef __attribute__((address_space(3))) void* lds_t;
  __builtin_amdgcn_global_load_lds((gbl_t)(p), (lds_t)lds, 16, 0, 0);
}

// Waits until at most VM vector memory instructions (which complete in
// order) and no LDS reads of this wave are outstanding.
template <int VM>
__device__ __forceinline__ void wait_counts() {
  static_assert(VM < 64, "vmcnt has 6 bits");
  // vmcnt 3:0 and 15:14, expcnt 6:4 (not waited for), lgkmcnt 11:8
  __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | 0x70);
}

// Workgroup barrier of the operand pipeline; the waits before it are the
// callers'.
__device__ __forceinline__ void pipe_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

static __device__ const u32x4_t kZeroPage[1] = {{0, 0, 0, 0}};

// The lane id, hidden from the optimiser: what is derived from it is computed
// where it is used instead of being kept in registers from tile to tile.
__device__ __forceinline__ int opaque_lane() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}

template <int N>
using Int = std::integral_constant<int, N>;
// f(Int<I>{}), ..., f(Int<N - 1>{})
template <int I, int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(Int<I>{});
    static_for<I + 1, N>(f);
  }
}

template <bool PKS, bool QKS, int BM_, int BN_, int WM_, int BK_, int NS_>
struct DmaCore {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = 4 / WM_, BK = BK_, NS = NS_;
  static constexpr int MI = BM / (32 * WM), NJ = BN / (32 * WN), SK = BK / 16;
  static constexpr int PB = BM * BK * 2, QB = BN * BK * 2;  // bytes of a stage's tiles
  static constexpr int NP = PB / 4096, NQ = QB / 4096;      // DMA per wave and stage
  static constexpr int kSlotBytes = PB + QB;
  static constexpr bool kGrid = true;  // rows on the 16-byte grid
  static constexpr bool kWhole = NS == 2;  // run(): a stage's fragments in registers
  static constexpr int kLdsBytes = kSlotBytes;  // of lds()
  // waves per SIMD: what the LDS allows of workgroups per CU
  static constexpr int kWaves = 160 * 1024 / (NS * kSlotBytes) < 3 ? 160 * 1024 / (NS * kSlotBytes) : 3;
  static_assert(BK == 64 || (BK == 32 && !kWhole), "a stage of two slots is four k steps");
  static_assert(PB % 4096 == 0 && QB % 4096 == 0, "whole DMA instructions for four waves");

  template <int S>
  static __device__ __forceinline__ char* slot() {
    __shared__ __attribute__((aligned(1024))) char mem[kSlotBytes];
    return mem;
  }
  // scratch for a result
  static __device__ __forceinline__ char* lds() { return slot<0>(); }

  // One operand: R rows (or columns), lane offsets of this wave's DMA.
  template <bool KS, int R>
  struct Operand {
    static constexpr int N = R * BK * 2 / 4096;
    const char* base;  // of stage 0
    int64_t step;      // bytes from one stage to the next
    uint32_t off[N];
    // first k, within a stage, of the 16 bytes lane `lane` copies in the
    // tile's i-th KiB
    static __device__ __forceinline__ int k_of(int i, int lane) {
      if constexpr (KS) {
        constexpr int LR = R / 8;
        return i * (64 / LR) + lane / LR;
      } else {
        constexpr int LR = BK / 8;
        const int r = i * (64 / LR) + lane / LR;
        return 8 * ((lane % LR) ^ (BK == 64 ? (r >> 1) & 7 : (r >> 2) & 3));
      }
    }
    __device__ __forceinline__ void init(const uint16_t* p, int64_t ld, int n, int wave, int lane) {
      base = reinterpret_cast<const char*>(p);
      step = KS ? ld * BK * 2 : BK * 2;
#pragma unroll
      for (int d = 0; d < N; ++d) {
        const int i = wave * N + d;
        const int k = k_of(i, lane);
        if constexpr (KS) {
          constexpr int LR = R / 8;
          const int sw = R >= 128 ? k & 3 : R == 64 ? (k >> 1) & 1 : 0;
          const int c = 8 * ((lane % LR) ^ (sw << 2));
          off[d] = static_cast<uint32_t>((k * ld + (c < n ? c : 0)) * 2);
        } else {
          const int r = i * (512 / BK) + lane / (BK / 8);
          off[d] = static_cast<uint32_t>(((r < n ? r : n - 1) * ld + k) * 2);
        }
      }
    }
    // piece D of the stage that starts at k = kf BK and holds kleft k; the
    // rest of it is zero
    template <int D>
    __device__ __forceinline__ void issue_tail(int64_t kf, char* tile, int wave, int lane,
                                               int kleft) const {
      const char* p = k_of(wave * N + D, lane) < kleft ? base + kf * step + off[D]
                                   : reinterpret_cast<const char*>(kZeroPage);
      dma16_at(p, tile + (wave * N + D) * 1024);
    }
  };

  // LDS byte offset of this lane's part of the fragment of block b, k step
  // g: K-contiguous one 16-byte read; K-strided two transposed reads, the
  // second 4 k rows on.
  template <bool KS, int R>
  static __device__ __forceinline__ bf16x8_t frag(const char* tile, int row0, int b, int g,
                                                  int lane) {
    if constexpr (KS) {
      const int s = lane & 15, kk = s >> 2;  // k % 4 of the row this lane addresses
      const int q = (row0 >> 5) + b;
      const int sw = R >= 128 ? kk : R == 64 ? kk >> 1 : 0;
      const int kr = 8 * (lane >> 5) + kk;
      const char* a = tile + (kr * R + ((q ^ sw) << 5) + 16 * ((lane >> 4) & 1) + 4 * (s & 3)) * 2 +
                      g * 16 * R * 2;
      const s16x4_t lo = lds_read_tr(reinterpret_cast<const uint16_t*>(a));
      const s16x4_t hi = lds_read_tr(reinterpret_cast<const uint16_t*>(a + 4 * R * 2));
      return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const int r = row0 + (lane & 31);  // blocks are 32 rows: the same swizzle
      const int sw = BK == 64 ? (r >> 1) & 7 : (r >> 2) & 3;
      const int c = (2 * g + (lane >> 5)) ^ sw;
      return *reinterpret_cast<const bf16x8_t*>(tile + (r * BK + 8 * c) * 2 + b * 32 * BK * 2);
    }
  }

  struct Frags {
    bf16x8_t p[MI], q[NJ];
  };

  static constexpr int DPS = NP + NQ;  // a wave's DMA instructions per stage

  template <bool ADD = false>
  static __device__ __forceinline__ void run(const TileArgs<uint16_t>& w,
                                             f32x16_t (&acc)[NJ][MI]) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ri = (wave % WM) * 32 * MI, rj = (wave / WM) * 32 * NJ;
    if constexpr (!ADD) zero_acc(acc);
    if (w.K <= 0) return;
    Operand<PKS, BM> po;
    Operand<QKS, BN> qo;
    po.init(w.P, w.ldp, w.pn, wave, lane);
    qo.init(w.Q, w.ldq, w.qn, wave, lane);
    // stage 0 is the sum's ragged end, if it has one; the others are whole,
    // and stage kt starts at k = (kt + shift) BK
    const int kleft = w.K % BK, nk = w.K / BK + (kleft != 0);
    const int shift = kleft != 0 ? -1 : 0;

    // DMA instruction D (P's first) of a whole stage
    auto issue1 = [&](int kt, auto slot_c, auto d_c) {
      char* tile = slot<decltype(slot_c)::value>();
      constexpr int d = decltype(d_c)::value;
      if constexpr (d < NP)
        dma16(po.base + (kt + shift) * po.step, po.off[d], tile + (wave * NP + d) * 1024);
      else
        dma16(qo.base + (kt + shift) * qo.step, qo.off[d - NP],
              tile + PB + (wave * NQ + d - NP) * 1024);
    };
    auto issue = [&](int kt, auto slot_c) {
      static_for<0, DPS>([&](auto d_c) { issue1(kt, slot_c, d_c); });
    };
    // This wave's DMA of a stage has landed when at most that of the newer
    // stages is outstanding; behind the barrier, everybody's has.
    auto landed = [&](int newer) {
      static_for<0, NS - 1>([&](auto i_c) {
        constexpr int i = decltype(i_c)::value;
        if (i == NS - 2 ? newer >= i : i == 0 ? newer <= 0 : newer == i) wait_counts<i * DPS>();
      });
    };

    if (kleft != 0) {
      const int64_t kf = w.K / BK;
      static_for<0, NP>([&](auto d) {
        po.template issue_tail<decltype(d)::value>(kf, slot<0>(), wave, lane, kleft);
      });
      static_for<0, NQ>([&](auto d) {
        qo.template issue_tail<decltype(d)::value>(kf, slot<0>() + PB, wave, lane, kleft);
      });
    } else {
      issue(0, Int<0>{});
    }
    static_for<1, NS>([&](auto s) {
      if (decltype(s)::value < nk) issue(decltype(s)::value, s);
    });
    if (nk >= NS) wait_counts<(NS - 1) * DPS>();
    else wait_counts<0>();
    pipe_barrier();

    auto read = [&](Frags& fr, auto slot_c, int g, auto r_c) {
      constexpr int r = decltype(r_c)::value;
      const char* tile = slot<decltype(slot_c)::value>();
      if constexpr (r < MI) fr.p[r] = frag<PKS, BM>(tile, ri, r, g, lane);
      else fr.q[r - MI] = frag<QKS, BN>(tile + PB, rj, r - MI, g, lane);
    };
    auto mfma = [&](Frags& fr, auto m_c) {
      constexpr int m = decltype(m_c)::value;
      acc[m / MI][m % MI] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          fr.q[m / MI], fr.p[m % MI], acc[m / MI][m % MI], 0, 0, 0);
    };
    constexpr int M = MI * NJ, R = MI + NJ;  // MFMAs and fragments of a k step

    if constexpr (kWhole) {
      // Two slots of four k steps, the fragments of a whole stage in
      // registers.  A slot is read in two steps' time (the last step of the
      // stage before and the first of its own) and then free: the DMA of stage
      // kt + 2 goes out in step 1 of stage kt and is needed in step 3 of stage
      // kt + 1, six k steps later.  With fragments of two steps only, a slot
      // is free behind step 2 and the DMA has four.  The two measured, us:
      // loss 4096 x 163840 x 7168 (256 x 256) 7185 against 7340, experts'
      // products 65536 rows of 128 (256 x 256 NT) 2155 against 2214, 700 rows
      // of 20 (128 x 128 NN) 13.4 against 16.4, loss 33 x 32000 x 2048 30.5
      // against 32.7, 1024 x 50048 x 1024 113 against 115.
      Frags f[4];
      constexpr int RM = M * 3 / 4;  // reads are spread over the first RM MFMAs
      static_for<0, R>([&](auto r) { read(f[0], Int<0>{}, 0, r); });
      static_for<0, R>([&](auto r) { read(f[1], Int<0>{}, 1, r); });
      auto reads = [&](auto slot_c, auto g_c, auto m_c) {
        constexpr int m = decltype(m_c)::value, g = decltype(g_c)::value;
        if constexpr (m < RM)
          static_for<m * 2 * R / RM, (m + 1) * 2 * R / RM>([&](auto i_c) {
            constexpr int i = decltype(i_c)::value;
            read(f[g + i / R], slot_c, g + i / R, Int<i % R>{});
          });
      };
      auto stage = [&](int kt, auto slot_c, auto steady_c) {
        constexpr int S = decltype(slot_c)::value;
        constexpr bool STEADY = decltype(steady_c)::value;
        static_for<0, M>([&](auto m_c) {
          mfma(f[0], m_c);
          reads(slot_c, Int<2>{}, m_c);
          __builtin_amdgcn_sched_barrier(0);
        });
        wait_counts<63>();  // this wave has read the slot
        pipe_barrier();     // so has everybody
        if constexpr (!STEADY) {
          if (kt + 2 < nk) issue(kt + 2, slot_c);
        }
        __builtin_amdgcn_sched_barrier(0);
        static_for<0, M>([&](auto m_c) {
          constexpr int m = decltype(m_c)::value;
          mfma(f[1], m_c);
          if constexpr (STEADY)
            static_for<m * DPS / M, (m + 1) * DPS / M>(
                [&](auto d_c) { issue1(kt + 2, slot_c, d_c); });
          __builtin_amdgcn_sched_barrier(0);
        });
        static_for<0, M>([&](auto m_c) {
          mfma(f[2], m_c);
          __builtin_amdgcn_sched_barrier(0);
        });
        if (STEADY || kt + 2 < nk) wait_counts<DPS>();
        else wait_counts<0>();
        pipe_barrier();  // the next stage is whole
        __builtin_amdgcn_sched_barrier(0);
        static_for<0, M>([&](auto m_c) {
          mfma(f[3], m_c);
          // (behind the last stage the reads find old data, which is not used)
          reads(Int<S ^ 1>{}, Int<0>{}, m_c);
          __builtin_amdgcn_sched_barrier(0);
        });
      };
      int kt = 0;
      for (; kt + 4 <= nk; kt += 2) {
        stage(kt, Int<0>{}, std::true_type{});
        stage(kt + 1, Int<1>{}, std::true_type{});
      }
      for (; kt < nk; kt += 2) {
        stage(kt, Int<0>{}, std::false_type{});
        if (kt + 1 < nk) stage(kt + 1, Int<1>{}, std::false_type{});
      }
    } else {
      Frags f[2];
      static_for<0, MI + NJ>([&](auto r) { read(f[0], Int<0>{}, 0, r); });

      // One stage: the matrix instructions of a k step run while the next
      // step's fragments are read.  Before the last step every wave has its
      // fragments of this stage and waits for the next stage's data; behind
      // the barrier the next stage is whole and this stage's slot is free, and
      // stage kt + NS goes into it.  STEADY: there is such a stage.
      auto stage = [&](int kt, auto slot_c, auto steady_c) {
        constexpr int S = decltype(slot_c)::value;
        constexpr bool STEADY = decltype(steady_c)::value;
        static_for<0, SK>([&](auto g_c) {
          constexpr int g = decltype(g_c)::value;
          constexpr bool last = g == SK - 1;
          Frags& cur = f[g & 1];
          Frags& nxt = f[(g + 1) & 1];
          if constexpr (last) {
            if constexpr (STEADY) wait_counts<(NS - 2) * DPS>();
            else landed(nk - 2 - kt);
            pipe_barrier();
            if constexpr (!STEADY) {
              if (kt + NS < nk) issue(kt + NS, slot_c);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
          static_for<0, MI * NJ>([&](auto m_c) {
            constexpr int m = decltype(m_c)::value;
            acc[m / MI][m % MI] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                cur.q[m / MI], cur.p[m % MI], acc[m / MI][m % MI], 0, 0, 0);
            // (behind the last stage the reads find old data, which is not used)
            constexpr int RM = MI * NJ < MI + NJ ? MI * NJ : MI + NJ;
            if constexpr (m < RM)
              static_for<m * (MI + NJ) / RM, (m + 1) * (MI + NJ) / RM>([&](auto r_c) {
                if constexpr (!last) read(nxt, slot_c, g + 1, r_c);
                else read(nxt, Int<(S + 1) % NS>{}, 0, r_c);
              });
            // the refill's DMA spread over the step's second part
            if constexpr (last && STEADY) {
              constexpr int M0 = MI + NJ < MI * NJ ? MI + NJ : 0, MS = MI * NJ - M0;
              if constexpr (m >= M0)
                static_for<(m - M0) * DPS / MS, (m - M0 + 1) * DPS / MS>(
                    [&](auto d_c) { issue1(kt + NS, slot_c, d_c); });
            }
            __builtin_amdgcn_sched_barrier(0);
          });
        });
      };
      static_assert(SK % 2 == 0, "fragment buffers alternate evenly over a stage");
      int kt = 0;
      for (; kt + 2 * NS <= nk; kt += NS)
        static_for<0, NS>([&](auto s) { stage(kt + decltype(s)::value, s, std::true_type{}); });
      for (; kt < nk; kt += NS)
        static_for<0, NS>([&](auto s) {
          if (kt + decltype(s)::value < nk)
            stage(kt + decltype(s)::value, s, std::false_type{});
        });
    }
  }

  // C[i][j] = acc (+ add[i][j]) for i < rows, j < cols.  add may be C.  The
  // rows of C and add are on the 16-byte grid and cols is a multiple of 8.
  // Each wave turns its accumulators into rows in LDS (16-byte chunk c of row
  // i at c ^ i, in the low bits) and stores 16 bytes a lane along the rows:
  // values already in the storage type, or fp32 where something is added.
  // STREAM: nontemporal stores (stream_gradient).
  template <bool STREAM = false, typename TO, typename TA>
  static __device__ __forceinline__ void write(f32x16_t (&acc)[NJ][MI], TO* C, int64_t ldc,
                                               const TA* add, int64_t lda, int rows, int cols) {
    if (sizeof(TO) == 2 && add == nullptr) rows_out<STREAM, true>(acc, C, ldc, add, lda, rows, cols);
    else rows_out<STREAM, false>(acc, C, ldc, add, lda, rows, cols);
  }

  // Bytes of a staged row: up to 256, as many as leave each wave a region in
  // the slots.  (Behind the last barrier of run() no wave reads operands any
  // more, so the slots are free.)
  static constexpr int stage_row(int bytes) {
    int rb = bytes < 256 ? bytes : 256;
    while (kSlotBytes / (32 * MI * rb) * NS < 4) rb /= 2;
    return rb;
  }
  // HALF: staged as bf16, else as fp32
  template <bool STREAM, bool HALF, typename TO, typename TA>
  static __device__ __forceinline__ void rows_out(f32x16_t (&acc)[NJ][MI], TO* C, int64_t ldc,
                                                  const TA* add, int64_t lda, int rows, int cols) {
    constexpr int ES = HALF ? 2 : 4;
    constexpr int RB = stage_row(NJ * 32 * ES);
    constexpr int CW = RB / ES, JB = CW / 32;  // columns of a staged row, blocks of 32
    constexpr int NCH = RB / 16, SH = NCH == 16 ? 0 : NCH == 8 ? 1 : 2;
    constexpr int REGION = 32 * MI * RB, PER = kSlotBytes / REGION;
    static_assert(PER >= 1 && PER * NS >= 4 && NJ % JB == 0, "a region for each wave");
    const int lane = opaque_lane();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    char* S = slot<0>();
    static_for<1, NS>([&](auto s) {
      if (wave / PER == decltype(s)::value) S = slot<decltype(s)::value>();
    });
    S += wave % PER * REGION;
    const int i0 = (wave % WM) * 32 * MI, j0 = (wave / WM) * 32 * NJ;
    const int fr = lane & 31, hl = lane >> 5;
    auto chunk = [&](int i, int c) { return S + i * RB + ((c ^ ((i >> SH) & (NCH - 1))) << 4); };
#pragma unroll
    for (int h = 0; h < NJ / JB; ++h) {
#pragma unroll
      for (int b = 0; b < JB; ++b)
#pragma unroll
        for (int bi = 0; bi < MI; ++bi)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x16_t& a = acc[h * JB + b][bi];
            const int i = 32 * bi + fr;
            if constexpr (HALF) {
              *reinterpret_cast<u32x2_t*>(chunk(i, 4 * b + q) + 8 * hl) =
                  u32x2_t{pack_bf16(a[4 * q], a[4 * q + 1]), pack_bf16(a[4 * q + 2], a[4 * q + 3])};
            } else {
              *reinterpret_cast<f32x4_t*>(chunk(i, 8 * b + 2 * q + hl)) =
                  f32x4_t{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
            }
          }
      // the wave's own region: its LDS accesses complete in order
      wave_sync();
      constexpr int LC = ES == 2 || sizeof(TO) == 4 ? NCH : NCH / 2;  // lanes to a row
      constexpr int LR = 64 / LC;                                     // rows at a time
      const int c = lane % LC, j = j0 + h * CW + c * (CW / LC);
      if (j < cols) {
#pragma unroll 8
        for (int r = lane / LC; r < 32 * MI; r += LR) {
          const int i = i0 + r;
          if (i >= rows) break;
          if constexpr (HALF) {
            put16<STREAM>(C + i * ldc + j, *reinterpret_cast<u32x4_t*>(chunk(r, c)));
          } else if constexpr (sizeof(TO) == 4) {
            f32x4_t v = *reinterpret_cast<f32x4_t*>(chunk(r, c));
            if (add != nullptr) {
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] += to_f32(add[i * lda + j + e]);
            }
            put16<STREAM>(C + i * ldc + j, v);
          } else {
            float v[8], o[8];
            __builtin_memcpy(v, chunk(r, 2 * c), 16);
            __builtin_memcpy(v + 4, chunk(r, 2 * c + 1), 16);
            load8(add + i * lda + j, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += o[e];
            store8<STREAM>(C + i * ldc + j, v);
          }
        }
      }
      wave_sync();
    }
  }
};

// The tile shapes of the DMA core.  Large: the least operand traffic for a
// flop (512 rows and columns of operands for 256 x 256 results), one
// workgroup to a CU, so nothing hides its prologue and epilogue.  Half and Medium: two workgroups
// to a CU.  Thin: a deep ring for streaming Q past a few rows of P.
// K-contiguous operands take 64 k a stage, whole 128-byte lines; K-strided
// ones always read whole lines and take 32, which doubles the stages in
// flight.  Large NN (one of each) measured 2147 us with 32 k and 2200 with
// 64 (65536 rows, 128 experts of 7168 x 2048).
template <bool PKS, bool QKS>
using LargeCore = DmaCore<PKS, QKS, 256, 256, 2, (PKS || QKS) ? 32 : 64, (PKS || QKS) ? 4 : 2>;
template <bool PKS, bool QKS>
using HalfCore = DmaCore<PKS, QKS, 128, 256, 2, 32, 3>;
template <bool PKS, bool QKS>
using MediumCore = DmaCore<PKS, QKS, 128, 128, 2, 64, 2>;
template <bool PKS, bool QKS>
using ThinCore = DmaCore<PKS, QKS, 32, 128, 1, 64, 6>;

// Which of them: the least estimated time on 256 CUs.  A workgroup takes
// stage x K / 64 + fixed microseconds, where the time of 64 k grows from
// `alone` to `full` with the number of workgroups that share the GPU (matrix
// cores of their CU, memory); tiles beyond one a place take further rounds,
// the last with the time of the tiles that are left for it (counting it as a
// whole one keeps 8192 rows of 16 experts, 1000 x 1416 (TN), 2048 of 8, 2048 x
// 1408 (TN), and 8192 of 16, 1024 x 2048 (NT), from the better tiles: 34.4, 21.5
// and 47.5 us against 39.7, 23.8 and 50.2).  The constants are fits to measured
// products of 8 to 65536 rows, 1 to 128 experts, sides 1000 to 7168 and 32000
// to 163840 vocabulary rows; some of what they rest on (us, shape by shape):
//   8 rows x 64 experts 2048x1408 (NN): Thin 12.1, Medium 17.2, Half 24.9, Large 38.8
//   700 rows x 20 experts 1280x1024 (NN): Medium 13.5, Thin 14.5, Half 18.9, Large 27.9
//   8192 rows x 16 experts 1000x1416 (TN): Half 32, Medium 37.5, Large 39
//   2000 rows x 1 expert 1024x4096 (TN): Medium 20.4, Half 24.9
//   loss 1024 x 50048 x 1024 (NT): Medium 115, Half 118, Large 133, Thin 356
//   loss 4096 x 163840 x 7168 (NT): Large 7240, Medium 8700, Half 9720
struct ShapeCost {
  int bm, bn, per_cu;
  double alone, full, fixed;
};
inline double shape_time(const ShapeCost& c, double row_tiles, int64_t cols, int64_t k) {
  const double tiles = row_tiles * static_cast<double>((cols + c.bn - 1) / c.bn);
  const double places = 256.0 * c.per_cu;
  auto round = [&](double n) {  // n workgroups
    const double load = std::fmin(1.0, std::fmax(0.0, (n - 128.0) / (places - 128.0)));
    return static_cast<double>(k) / 64.0 * (c.alone + (c.full - c.alone) * load) + c.fixed;
  };
  if (tiles >= 8.0 * places) return (tiles / places + 0.5) * round(places);
  const double whole = std::floor(tiles / places), rest = tiles - whole * places;
  return whole * round(places) + (rest > 0.0 ? round(rest) : 0.0);
}
enum Shape { kLarge, kHalf, kMedium, kThin };
constexpr ShapeCost kShapeNT[] = {{256, 256, 1, 1.40, 1.72, 12.0}, {128, 256, 2, 1.40, 2.45, 4.0},
                                  {128, 128, 2, 0.50, 1.12, 3.0}, {32, 128, 1, 0.30, 0.80, 2.0}};
constexpr ShapeCost kShapeNN[] = {{256, 256, 1, 1.50, 1.79, 12.0}, {128, 256, 2, 1.10, 2.15, 3.0},
                                  {128, 128, 2, 0.50, 1.13, 3.0}, {32, 128, 1, 0.30, 0.80, 2.0}};
constexpr ShapeCost kShapeTN[] = {{256, 256, 1, 1.45, 1.65, 9.0}, {128, 256, 2, 1.05, 2.10, 4.2},
                                  {128, 128, 2, 0.55, 1.20, 3.4}};
// the core for any operands: 128 x 128, 64 x 64
constexpr ShapeCost kShapeAnyBf16[] = {{128, 128, 2, 1.20, 1.85, 3.0}, {64, 64, 4, 0.70, 1.60, 2.0}};
constexpr ShapeCost kShapeAnyFp32[] = {{128, 128, 2, 3.80, 5.80, 6.0}, {64, 64, 4, 1.80, 4.10, 2.5}};
// rows(bm): row tiles of bm rows
template <int N, typename R>
Shape pick_shape(const ShapeCost (&c)[N], R&& rows, int64_t cols, int64_t k) {
  int best = 0;
  double t = 0.0;
  for (int i = 0; i < N; ++i) {
    const double e = shape_time(c[i], rows(c[i].bm), cols, k);
    if (i == 0 || e < t) {
      best = i;
      t = e;
    }
  }
  return static_cast<Shape>(best);
}

// Whether the core for any operands takes its 128x128 tiles.
template <typename T, typename R>
bool pick_any_large(R&& rows, int64_t cols, int64_t k) {
  return pick_shape(sizeof(T) == 2 ? kShapeAnyBf16 : kShapeAnyFp32, rows, cols, k) == 0;
}

// Whether the DMA core stores a weight gradient of rows x cols past the caches,
// which leaves them to the operands; the optimizer step reads it after the
// whole backward.  us with and without, bf16:
//   rows of whole 128-byte lines: 4096 rows of 64 experts, 2048 x 1408, 76 and
//   103; 65536 of 128, 7168 x 2048, 2220 and 2308; 700 of 20, 1280 x 1024, 14.2
//   and 14.8; loss 1024 x 50048 x 1024, backward 610 and 625
//   others pay for the parts of lines: 4096 of 16, 1024 x 1000 (33 MB), 24.6 and
//   17.6; 8192 of 16, 2000 x 1032 (66 MB), 56.8 and 55.6; 20000 of 16, 2040 x
//   2056 (134 MB), 198 and 218
// Not activations, which the next call reads: a product and the one after it,
// 10000 rows of 16 experts, 1024 x 2816, take 140 with it and 132 without.
template <typename TO>
bool stream_gradient(const TO* p, int64_t rows, int64_t cols) {
  const int64_t line = cols * static_cast<int64_t>(sizeof(TO));
  return (line % 128 == 0 && reinterpret_cast<uintptr_t>(p) % 128 == 0) ||
         rows * line >= (int64_t{128} << 20);
}

// The core of operands that the DMA core does not take.
template <typename T, bool PKS, bool QKS, int B>
using OtherCore = std::conditional_t<sizeof(T) == 4, SplitCore<PKS, QKS, B>, AnyCore<T, PKS, QKS, B>>;

}  // namespace muon
