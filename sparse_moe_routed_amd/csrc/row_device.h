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

// 16-byte chunk c of a row of H elements, zeros past its end.  ODD: H is no
// multiple of VEC, so the last chunk is taken element by element.
template <class A, bool ODD>
__device__ __forceinline__ u32x4_t load_chunk(const typename A::T* row, int c, int H) {
  constexpr int V = A::VEC;
  if constexpr (!ODD) {
    return c * V < H ? ld16(row + c * V) : u32x4_t{0u, 0u, 0u, 0u};
  } else {
    if ((c + 1) * V <= H) return *reinterpret_cast<const u32x4_e2*>(row + c * V);
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = c * V + i < H ? A::get(row[c * V + i]) : 0.f;
    return A::pack(v);
  }
}

template <class A, bool ODD>
__device__ __forceinline__ void store_chunk(typename A::T* row, int c, int H,
                                            const float (&v)[A::VEC]) {
  constexpr int V = A::VEC;
  if constexpr (!ODD) {
    if (c * V < H) *reinterpret_cast<u32x4_t*>(row + c * V) = A::pack(v);
  } else {
    if ((c + 1) * V <= H) {
      *reinterpret_cast<u32x4_e2*>(row + c * V) = A::pack(v);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c * V + i < H) row[c * V + i] = A::put(v[i]);
    }
  }
}

// Sums of one or two values per thread over the threads of a row, in a fixed
// association, the results in every thread.  WAVE: the row is one wave; else
// it is the whole workgroup, and `slot` is one float (2) per wave in LDS that
// no other reduction uses until the next barrier after this one.
template <bool WAVE>
__device__ __forceinline__ float row_sum(float v, float* slot) {
  v = wave_sum_f32(v);
  if constexpr (!WAVE) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slot[0];
    for (unsigned i = 1; i < blockDim.x >> 6; ++i) v += slot[i];
  }
  return v;
}

template <bool WAVE>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* slot) {
  float2 v = make_float2(wave_sum_f32(a), wave_sum_f32(b));
  if constexpr (!WAVE) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slot[0];
    for (unsigned i = 1; i < blockDim.x >> 6; ++i) {
      v.x += slot[i].x;
      v.y += slot[i].y;
    }
  }
  return v;
}

__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + expf(-g));
}

// Full gates of the norm kernels (a token gate is a factor of the whole row)
constexpr int kGateRow = 0, kGateFull = 1, kGateFullSigmoid = 2;

}  // namespace moe
