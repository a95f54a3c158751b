// Helpers shared by the operators that write gradients for the optimizer
// step: the embedding (embed.hip), the vocabulary loss (lm_loss.hip) and
// the expert products (experts.hip).
#pragma once

#include <string>

#include "muon.h"
#include "muon_internal.h"

namespace muon {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// two floats -> packed bf16 pair, round to nearest even (v_cvt_pk_bf16_f32)
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}

// Orders a wave's LDS accesses before and after it (the lanes of a wave run
// in step and its LDS accesses complete in order).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Storage types: float, or uint16_t holding a bf16 pattern.
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(uint16_t x) { return bf16_to_f32(x); }
__device__ __forceinline__ void from_f32(float x, float* p) { *p = x; }
__device__ __forceinline__ void from_f32(float x, uint16_t* p) { *p = f32_to_bf16(x); }

// 8 consecutive elements <-> 8 floats, any element alignment (gfx950 global
// accesses need none; aligned ones are faster).
__device__ __forceinline__ void load8(const uint16_t* p, float* o) {
  u32x4_t w;
  __builtin_memcpy(&w, p, 16);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    o[2 * k] = __uint_as_float(w[k] << 16);
    o[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float* o) {
  __builtin_memcpy(o, p, 32);
}
// Stores a 16-byte vector; STREAM: not to be kept in the caches (p aligned).
template <bool STREAM, typename V>
__device__ __forceinline__ void put16(void* p, V v) {
  static_assert(sizeof(V) == 16, "");
  if constexpr (STREAM) __builtin_nontemporal_store(v, static_cast<V*>(p));
  else __builtin_memcpy(p, &v, 16);
}
template <bool STREAM = false>
__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
  put16<STREAM>(p, u32x4_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                           pack_bf16(v[6], v[7])});
}
template <bool STREAM = false>
__device__ __forceinline__ void store8(float* p, const float* v) {
  put16<STREAM>(p, f32x4_t{v[0], v[1], v[2], v[3]});
  put16<STREAM>(p + 4, f32x4_t{v[4], v[5], v[6], v[7]});
}

// ---- host side ----

inline bool train_dtype_ok(int32_t d) { return d == MUON_DTYPE_FP32 || d == MUON_DTYPE_BF16; }
inline size_t train_dtype_size(int32_t d) { return d == MUON_DTYPE_FP32 ? 4 : 2; }
// Positions are 32-bit in the kernels.
constexpr int64_t kMaxTokens = (static_cast<int64_t>(1) << 26) - 1;
constexpr int64_t kMaxVocab = (static_cast<int64_t>(1) << 31) - 2;
constexpr int64_t kMaxDim = static_cast<int64_t>(1) << 22;

inline int check_token_sizes(int64_t n, int64_t vocab, int64_t dim) {
  if (n < 0 || n > kMaxTokens) return set_error(MUON_ERR_BAD_SHAPE, "n must be in [0, 2^26)");
  if (vocab < 1 || vocab > kMaxVocab)
    return set_error(MUON_ERR_BAD_SHAPE, "vocab must be in [1, 2^31 - 2]");
  if (dim < 1 || dim > kMaxDim) return set_error(MUON_ERR_BAD_SHAPE, "dim must be in [1, 2^22]");
  return MUON_OK;
}
// On the 16-byte grid, for every type: base, row stride and row length.  The
// row stride also keeps a tile's lane offsets within 32 bits.
inline bool on_grid(const void* p, int64_t ld, int64_t cols) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0 && cols % 8 == 0 &&
         ld <= (1 << 22);
}
inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

inline int check_launch(const char* what) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? MUON_OK : set_hip_error(e, what);
}

}  // namespace muon
