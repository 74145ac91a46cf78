// Device helpers of the row kernels (norms, dispatch, their gradients): a row
// of H features is handled in 16-byte chunks, VEC elements each.
#pragma once

#include "moe_device.h"

namespace moe {

// Chunks of rows whose length is no multiple of VEC start at any element:
// global memory takes 16-byte accesses at element alignment.
typedef u32x4_t u32x4_e2 __attribute__((aligned(2)));

struct RowBf16 {
  typedef uint16_t T;
  static constexpr int VEC = 8;
  static __device__ __forceinline__ float get(uint16_t v) { return bf16_to_f32(v); }
  // round to nearest even, NaN stays NaN (v_cvt_pk_bf16_f32)
  static __device__ __forceinline__ uint16_t put(float v) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  }
  static __device__ __forceinline__ void unpack(u32x4_t r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(r[i] << 16);
      v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ u32x4_t pack(const float (&v)[8]) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    u32x4_t r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bf16x2_t p = {static_cast<__bf16>(v[2 * i]), static_cast<__bf16>(v[2 * i + 1])};
      r[i] = __builtin_bit_cast(uint32_t, p);
    }
    return r;
  }
};

struct RowF32 {
  typedef float T;
  static constexpr int VEC = 4;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
  static __device__ __forceinline__ void unpack(u32x4_t r, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
  }
  static __device__ __forceinline__ u32x4_t pack(const float (&v)[4]) {
    u32x4_t r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(v[i]);
    return r;
  }
};

// Sum of one value per thread over the NT threads of a row (NT = 64: one
// wave; else the whole workgroup, through `slot`, NT / 64 floats of LDS that
// no other reduction uses until the next barrier after this one).  Fixed
// association, the result in every thread.
template <int NT>
__device__ __forceinline__ float row_sum(float v, float* slot) {
  v = wave_sum_f32(v);
  if constexpr (NT > kWave) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slot[0];
#pragma unroll
    for (int i = 1; i < NT / kWave; ++i) v += slot[i];
  }
  return v;
}

__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + expf(-g)); }

}  // namespace moe
