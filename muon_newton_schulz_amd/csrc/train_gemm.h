// Tile cores of the matrix products behind the vocabulary loss
// (lm_loss.hip) and the expert products (experts.hip).
//
// A core computes one output tile C[i][j] = sum_k P(i, k) Q(j, k), i < BM,
// j < BN, with four waves in a WM x WN grid, each MI x NJ blocks of 32x32
// on the matrix cores with fp32 accumulation.  An operand is K-contiguous
// (element (r, k) at p[r * ld + k]) or K-strided (at p[k * ld + r]); pn and
// qn are the rows of P and Q that exist from the tile's first row on (the
// others count as zero and are not read), K the length of the sum.
//
// Accumulators (A operand = Q, B operand = P): acc[bj][bi][4 q + e] of a
// lane is element
//   i = wi * 32 MI + 32 bi + lane % 32,
//   j = wj * 32 NJ + 32 bj + 8 q + 4 (lane / 32) + e,
// so a lane holds four consecutive columns of one row.
#pragma once

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

// 8 k (bf16) or 4 k (fp32) of a 16-wide (8-wide) k step from LDS:
// transposed read of a K-strided tile.  Within each group of 16 lanes, lane
// l receives element l % 4 of the 8-byte blocks addressed by lanes
// 4 q + l / 4, q = 0..3.
__device__ __forceinline__ s16x4_t lds_read_tr(const uint16_t* p) {
  typedef __attribute__((address_space(3))) s16x4_t* lds_t;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)(p));
}

// ------------------------------------------------------------ any operands
//
// The core for operands off the 16-byte grid, and for fp32: 128x128 tiles,
// 64 bytes of k at a time (32 bf16, 16 fp32) through registers into
// double-buffered LDS, the next step's loads in flight during the current
// step's matrix instructions.  Loads need no alignment; a piece of 16 bytes
// that crosses the end of a row (or of the tile's columns) is read element
// by element, so nothing outside the operands is touched.
// fp32 runs on v_mfma_f32_32x32x2_f32: lane l of instruction s of a group
// of 8 k supplies k = 4 (l / 32) + s, for both operands.
template <typename T, bool PKS, bool QKS>
struct AnyCore {
  static constexpr int BM = 128, BN = 128, MI = 2, NJ = 2, WM = 2, WN = 2;
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr int E = 16 / sizeof(T);   // elements per 16-byte piece
  static constexpr int CK = 4 * E;           // k per step
  // LDS strides in elements.  K-contiguous rows of 64 bytes are padded to
  // 80, so that 16-byte reads of consecutive rows spread over the banks;
  // K-strided rows of 128 columns by 8 elements, so that the k rows the two
  // lane halves read differ by half the banks.
  static constexpr int SC = CK + E, SS = 128 + 8;
  static constexpr int kOperandBytes = 128 * SC * static_cast<int>(sizeof(T));  // >= CK * SS
  static_assert(CK * SS <= 128 * SC, "a K-strided tile fits the K-contiguous one's space");
  static constexpr int kLdsBytes = 4 * kOperandBytes;

  template <bool KS>
  static __device__ __forceinline__ u32x4_t piece(const T* p, int64_t ld, int n, int K, int k0,
                                                  int pc) {
    int r, k, left;
    const T* a;
    if (KS) {
      constexpr int PR = 128 / E;
      k = k0 + pc / PR;
      r = (pc % PR) * E;
      left = k < K ? n - r : 0;
      a = p + static_cast<int64_t>(k) * ld + r;
    } else {
      r = pc >> 2;
      k = k0 + (pc & 3) * E;
      left = r < n ? K - k : 0;
      a = p + static_cast<int64_t>(r) * ld + k;
    }
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
  template <bool KS>
  static __device__ __forceinline__ T* lds_piece(T* s, int pc) {
    constexpr int PR = 128 / E;
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

  static __device__ __forceinline__ void run(const T* P, int64_t ldp, int pn, const T* Q,
                                             int64_t ldq, int qn, int K,
                                             f32x16_t (&acc)[NJ][MI], char* smem) {
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int wi = wave % WM, wj = wave / WM;
    u32x4_t pr[2], qr[2];
    auto load = [&](int k0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        pr[h] = piece<PKS>(P, ldp, pn, K, k0, t + 256 * h);
        qr[h] = piece<QKS>(Q, ldq, qn, K, k0, t + 256 * h);
      }
    };
    auto buf = [&](int b, int op) {
      return reinterpret_cast<T*>(smem + (2 * b + op) * kOperandBytes);
    };
    auto store = [&](int b) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        *reinterpret_cast<u32x4_t*>(lds_piece<PKS>(buf(b, 0), t + 256 * h)) = pr[h];
        *reinterpret_cast<u32x4_t*>(lds_piece<QKS>(buf(b, 1), t + 256 * h)) = qr[h];
      }
    };
    zero_acc(acc);
    const int steps = (K + CK - 1) / CK;
    if (steps == 0) return;
    load(0);
    store(0);
    __syncthreads();
    for (int c = 0; c < steps; ++c) {
      const int b = c & 1;
      if (c + 1 < steps) load((c + 1) * CK);
      const T* ps = buf(b, 0);
      const T* qs = buf(b, 1);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        decltype(frag<PKS>(ps, 0, 0, 0)) p[MI];
        decltype(frag<QKS>(qs, 0, 0, 0)) q[NJ];
#pragma unroll
        for (int i = 0; i < MI; ++i) p[i] = frag<PKS>(ps, wi * 64 + 32 * i, g, lane);
#pragma unroll
        for (int j = 0; j < NJ; ++j) q[j] = frag<QKS>(qs, wj * 64 + 32 * j, g, lane);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            if constexpr (F32) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x2f32(q[j][e], p[i][e], acc[j][i], 0, 0, 0);
            } else {
              acc[j][i] =
                  __builtin_amdgcn_mfma_f32_32x32x16_bf16(q[j], p[i], acc[j][i], 0, 0, 0);
            }
          }
      }
      if (c + 1 < steps) store(b ^ 1);
      __syncthreads();
    }
  }
};

// Four consecutive columns of a row, `left` of which exist.
template <typename TO>
__device__ __forceinline__ void store_quad(TO* p, int left, f32x4_t v, bool add) {
  if (left <= 0) return;
  if (left >= 4) {
    if constexpr (sizeof(TO) == 4) {
      if (add) {
        f32x4_t o;
        __builtin_memcpy(&o, p, 16);
        v += o;
      }
      __builtin_memcpy(p, &v, 16);
    } else {
      if (add) {
        u32x2_t o;
        __builtin_memcpy(&o, p, 8);
        v += f32x4_t{__uint_as_float(o[0] << 16), __uint_as_float(o[0] & 0xffff0000u),
                     __uint_as_float(o[1] << 16), __uint_as_float(o[1] & 0xffff0000u)};
      }
      const u32x2_t w = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
      __builtin_memcpy(p, &w, 8);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < left) from_f32(add ? to_f32(p[e]) + v[e] : v[e], p + e);
  }
}

}  // namespace muon
