// Device helpers of the row kernels (norms, dispatch, their gradients): a row
// of H features is handled in 16-byte chunks, VEC elements each.
#pragma once

#include "moe_device.h"

namespace moe {

// Chunks of rows whose length is no multiple of VEC start at any element:
// global memory takes 16-byte accesses at element alignment.
typedef u32x4_t u32x4_e2 __attribute__((aligned(2)));

// A value of an input at a wave-uniform address, through the scalar cache: no
// output of a kernel overlaps its inputs, so the value cannot change.
template <typename T>
__device__ __forceinline__ T uniform_load(const T* p) {
  typedef const T __attribute__((address_space(4))) * const_ptr;
  return *(const_ptr)(reinterpret_cast<uintptr_t>(p));
}

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

// One row of a matrix, read and written in 16-byte chunks: chunk i * nt + tid
// by thread tid of nt.  Chunks past the row read as zeros and are not
// written.  The row must be uniform over the wave.  load_once is for data
// that this call reads once: with STREAM it does not stay in the caches
// (when that pays: streams_matrix, streams_slots in moe_internal.h).
//
// ODD == false (H a multiple of VEC): a raw buffer of the row's bytes, whose
// bounds check takes the place of a branch per chunk, with a scalar base and
// one offset register for all chunks (wide rows otherwise held a 64-bit
// address and a predicate per chunk and matrix, and spilled).
template <class A, bool ODD, bool STREAM>
struct RowRef {
  typedef typename A::T T;
  static constexpr int V = A::VEC;
  __amdgpu_buffer_rsrc_t rs;
  __device__ __forceinline__ RowRef(const void* m, size_t at, int H)
      : rs(__builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(static_cast<const T*>(m) + at), 0,
                                             H * static_cast<int>(sizeof(T)), 0x00020000)) {}
  // row r of m, or nothing at all (loads give zeros) for r < 0
  static __device__ __forceinline__ RowRef slot(const void* m, int r, int H) {
    RowRef ref(m, static_cast<size_t>(max(r, 0)) * H, r < 0 ? 0 : H);
    return ref;
  }
  __device__ __forceinline__ u32x4_t load(int i, int nt, int tid) const {
    return __builtin_amdgcn_raw_buffer_load_b128(rs, tid * 16, i * nt * 16, 0);
  }
  __device__ __forceinline__ u32x4_t load_once(int i, int nt, int tid) const {
    return __builtin_amdgcn_raw_buffer_load_b128(rs, tid * 16, i * nt * 16, STREAM ? 2 : 0);   // 2: nt
  }
  __device__ __forceinline__ void store(int i, int nt, int tid, const float (&v)[V]) const {
    store_raw(i, nt, tid, A::pack(v));
  }
  // The whole offset goes into the vector register.  With a scalar offset the
  // compiler puts no wait state between a 16-byte buffer store and the next
  // instruction, and where that one overwrote the data registers, some lanes
  // stored the new first word (seen now and then in 65536-wide float32 rows:
  // values of chunk i + 1 in chunk i).
  __device__ __forceinline__ void store_raw(int i, int nt, int tid, u32x4_t v) const {
    __builtin_amdgcn_raw_buffer_store_b128(v, rs, (i * nt + tid) * 16, 0, 0);
  }
};

// ODD: rows start at any element; the chunk that the row's end cuts is taken
// element by element.
template <class A, bool STREAM>
struct RowRef<A, true, STREAM> {
  typedef typename A::T T;
  static constexpr uint32_t V = A::VEC;
  T* row;
  uint32_t H;
  __device__ __forceinline__ RowRef(const void* m, size_t at, int len)
      : row(const_cast<T*>(static_cast<const T*>(m)) + at), H(len) {}
  __device__ __forceinline__ u32x4_t load(int i, int nt, int tid) const {
    const uint32_t h = static_cast<uint32_t>(i * nt + tid) * V;
    if (h + V <= H) return *reinterpret_cast<const u32x4_e2*>(row + h);
    float v[V];
#pragma unroll
    for (uint32_t e = 0; e < V; ++e) v[e] = h + e < H ? A::get(row[h + e]) : 0.f;
    return A::pack(v);
  }
  __device__ __forceinline__ u32x4_t load_once(int i, int nt, int tid) const {
    return load(i, nt, tid);
  }
  __device__ __forceinline__ void store(int i, int nt, int tid, const float (&v)[V]) const {
    const uint32_t h = static_cast<uint32_t>(i * nt + tid) * V;
    if (h + V <= H) {
      *reinterpret_cast<u32x4_e2*>(row + h) = A::pack(v);
    } else {
#pragma unroll
      for (uint32_t e = 0; e < V; ++e)
        if (h + e < H) row[h + e] = A::put(v[e]);
    }
  }
};

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

// 1 / (1 + exp(-g)).  EXACT: expf; else exp2(-g log2 e), whose rounded
// argument costs |g| 2^-24 of the result: far below a bf16 rounding, and a
// third of the instructions.
template <bool EXACT>
__device__ __forceinline__ float sigmoid(float g) {
  const float e = EXACT ? expf(-g) : __builtin_amdgcn_exp2f(-1.44269504088896f * g);
  return __builtin_amdgcn_rcpf(1.0f + e);
}

// Rows and weights of a token's slots j0 .. j0 + 63, one per lane: row -1
// and weight 0 for a dropped pair (row outside [0, P)) and past slot k - 1.
// One vector load each; row(u) and weight(u) are scalars read from a lane
// where they are needed (a scalar load per slot took a round trip each, all
// of them up front took more scalar registers than there are).
template <bool WEIGHTED>
struct Slots {
  int r;
  float w;
  __device__ __forceinline__ Slots(const int32_t* pair_row, const float* weights, int j0, int k,
                                   int P) {
    const int j = j0 + (threadIdx.x & 63);
    r = j < k ? pair_row[j] : -1;
    w = 1.f;
    if constexpr (WEIGHTED) w = j < k ? weights[j] : 0.f;
    if (r < 0 || r >= P) r = -1;
    if (r < 0) w = 0.f;
  }
  __device__ __forceinline__ int row(int u) const { return __builtin_amdgcn_readlane(r, u); }
  __device__ __forceinline__ float weight(int u) const {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), u));
  }
};

// Full gates of the norm kernels (a token gate is a factor of the whole row)
constexpr int kGateRow = 0, kGateFull = 1, kGateFullSigmoid = 2;

}  // namespace moe
