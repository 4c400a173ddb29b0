// Row access shared by the memory-bound row kernels (sorted_rows.hip,
// block_norm.hip): 16-byte chunks of a row as fp32 values and back, and sums
// over the lanes of a wave.  Internal to libmoe.so.
#pragma once

#include "moe_common.h"

namespace moe {

// Elements of T in one 16-byte chunk.
template <typename T> constexpr int chunk_elems() { return 16 / (int)sizeof(T); }

__device__ __forceinline__ void unpack(u32x4_t v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(u32x4_t v, float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
}

// Two fp32 values as packed bf16, each rounded to nearest, ties to even (the
// hardware conversion of gfx950; NaN stays NaN).
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ u32x4_t pack(const float (&f)[8]) {
  u32x4_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  return v;
}
__device__ __forceinline__ u32x4_t pack(const float (&f)[4]) {
  u32x4_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(f[i]);
  return v;
}

// Sum of v over the 64 lanes of a wave, in every lane (all lanes active).
__device__ __forceinline__ float wave_sum_f32(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

// The routing weight of entry f, stored as bf16 or fp32.
__device__ __forceinline__ float weight_at(const void *w, bool is_bf16, int64_t f) {
  return is_bf16 ? to_f32(reinterpret_cast<const bf16_t *>(w)[f])
                 : reinterpret_cast<const float *>(w)[f];
}

}  // namespace moe
