// Device helpers of the row kernels (norms, dispatch, their gradients): a row
// of H features is handled in 16-byte chunks, VEC elements each.
#pragma once

#include "moe_device.h"

namespace moe {

// Chunks of bf16 rows of odd length start at any element: global memory takes
// 16-byte accesses at element alignment.
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
// EDGE says what the end of a row does to its last chunk.
constexpr int kEdgeWords = 0;   // whole chunks, or a cut that RowRef's bounds check handles
constexpr int kEdgeCut = 1;     // a cut between words, rows sharing a wave (PackRef)
constexpr int kEdgeOdd = 2;     // bf16 rows of odd length

// kEdgeWords (rows are whole 32-bit words: float32, bf16 of even length): a
// raw buffer of the row's bytes.  Its bounds check, word by word, takes the
// place of a branch per chunk, also for a chunk that the row's end cuts, with
// a scalar base for all chunks (wide rows otherwise held a 64-bit address and
// a predicate per chunk and matrix, and spilled).  Every access carries its
// whole offset in the vector register and the instruction: the check counts
// those, not the scalar offset, and chunks past the row have to fail it.
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
    return __builtin_amdgcn_raw_buffer_load_b128(rs, (i * nt + tid) * 16, 0, 0);
  }
  __device__ __forceinline__ u32x4_t load_once(int i, int nt, int tid) const {
    return __builtin_amdgcn_raw_buffer_load_b128(rs, (i * nt + tid) * 16, 0, STREAM ? 2 : 0);   // 2: nt
  }
  __device__ __forceinline__ void store(int i, int nt, int tid, const float (&v)[V]) const {
    store_raw(i, nt, tid, A::pack(v));
  }
  // A store has a second reason: with a scalar offset the compiler puts no
  // wait state between a 16-byte buffer store and the next instruction, and
  // where that one overwrote the data registers, some lanes stored the new
  // first word (seen now and then in 65536-wide float32 rows: values of chunk
  // i + 1 in chunk i).
  __device__ __forceinline__ void store_raw(int i, int nt, int tid, u32x4_t v) const {
    __builtin_amdgcn_raw_buffer_store_b128(v, rs, (i * nt + tid) * 16, 0, 0);
  }
};

// ODD: bf16 rows of odd length start at any element; the chunk that the row's
// end cuts is taken element by element, under a branch, so each chunk waits for
// its own loads (norm_in and its gradient, 4096 x 2559: 11.3 and 27.4 us a call;
// 2558: 9.6 and 19.8).
template <class A, bool STREAM>
struct RowRef<A, true, STREAM> {
  typedef typename A::T T;
  static constexpr uint32_t V = A::VEC;
  T* row;
  uint32_t H;
  bool on;
  // `on`: the row exists (it may differ between lanes); H is uniform
  __device__ __forceinline__ RowRef(const void* m, size_t at, int len, bool exists = true)
      : row(const_cast<T*>(static_cast<const T*>(m)) + at), H(len), on(exists) {}
  __device__ __forceinline__ u32x4_t load(int i, int nt, int tid) const {
    const uint32_t h = static_cast<uint32_t>(i * nt + tid) * V;
    if (on && h + V <= H) return *reinterpret_cast<const u32x4_e2*>(row + h);
    float v[V];
#pragma unroll
    for (uint32_t e = 0; e < V; ++e) v[e] = on && h + e < H ? A::get(row[h + e]) : 0.f;
    return A::pack(v);
  }
  __device__ __forceinline__ u32x4_t load_once(int i, int nt, int tid) const {
    return load(i, nt, tid);
  }
  __device__ __forceinline__ void store(int i, int nt, int tid, const float (&v)[V]) const {
    const uint32_t h = static_cast<uint32_t>(i * nt + tid) * V;
    if (!on) return;
    if (h + V <= H) {
      *reinterpret_cast<u32x4_e2*>(row + h) = A::pack(v);
    } else {
#pragma unroll
      for (uint32_t e = 0; e < V; ++e)
        if (h + e < H) row[h + e] = A::put(v[e]);
    }
  }
};

// A row of at most 32 chunks whose wave holds several: chunk `tid` of row t, a
// lane each, through a buffer of the whole matrix (of `rows` rows, under 2
// GiB).  Lanes past the row or the matrix have an offset past its end.  CUT:
// in the chunk that the row's end cuts, the next row's words are masked out
// of loads and left out of stores (norm_in, then its gradient, 131072 x 64
// bf16: 25.4 us without the masks, 27.2 with them).
template <class A, bool STREAM, bool CUT>
struct PackRef {
  typedef typename A::T T;
  static constexpr int V = A::VEC;
  static constexpr uint32_t kNowhere = 0x80000000u;
  __amdgpu_buffer_rsrc_t rs;
  uint32_t off;
  int words;        // of this lane's chunk inside the row
  int cut_words;    // of the cut chunk (uniform), 0 if there is none
  __device__ __forceinline__ PackRef(const void* m, int t, int rows, int H, int tid)
      : rs(__builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(m), 0,
                                             rows * H * static_cast<int>(sizeof(T)), 0x00020000)) {
    words = min(max(H - tid * V, 0), V) * static_cast<int>(sizeof(T)) / 4;
    cut_words = H % V * static_cast<int>(sizeof(T)) / 4;
    off = t < rows && words > 0 ? (t * H + tid * V) * static_cast<uint32_t>(sizeof(T)) : kNowhere;
  }
  template <int AUX>
  __device__ __forceinline__ u32x4_t get() const {
    u32x4_t r = __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, AUX);
    if constexpr (CUT)
#pragma unroll
      for (int e = 1; e < 4; ++e) r[e] = e < words ? r[e] : 0u;
    return r;
  }
  __device__ __forceinline__ u32x4_t load(int, int, int) const { return get<0>(); }
  __device__ __forceinline__ u32x4_t load_once(int, int, int) const { return get<STREAM ? 2 : 0>(); }
  __device__ __forceinline__ void store(int, int, int, const float (&v)[V]) const {
    const u32x4_t r = A::pack(v);
    __builtin_amdgcn_raw_buffer_store_b128(r, rs, !CUT || words == 4 ? off : kNowhere, 0, 0);
    if (!CUT) return;
    const uint32_t cut = words < 4 ? off : kNowhere;
    if (cut_words & 2) __builtin_amdgcn_raw_buffer_store_b64(u32x2_t{r[0], r[1]}, rs, cut, 0, 0);
    if (cut_words & 1)
      __builtin_amdgcn_raw_buffer_store_b32(cut_words & 2 ? r[2] : r[0], rs,
                                            cut + 4 * (cut_words & 2), 0, 0);
  }
};

// How a row kernel's threads share rows.  L: lanes of a row; 0: the row is a
// workgroup's, 64: a wave's, 8, 16 or 32: 64 / L rows share a wave.
template <int L>
struct RowShare {
  static constexpr bool WAVE = L != 0, PACK = WAVE && L < 64;
  static constexpr int ROWS = PACK ? 64 / L : 1;   // rows of a wave
  // a row's threads and this thread's place among them
  static __device__ __forceinline__ int threads() { return WAVE ? L : blockDim.x; }
  static __device__ __forceinline__ int place() { return WAVE ? threadIdx.x % L : threadIdx.x; }
  // this lane's row among the wave's
  static __device__ __forceinline__ int lane_row() { return PACK ? (threadIdx.x & 63) / L : 0; }
};

// Row t of a matrix with `rows` rows.
template <class A, int L, int EDGE, bool STREAM>
__device__ __forceinline__ auto row_ref(const void* m, int t, int rows, int H) {
  constexpr bool ODD = EDGE == kEdgeOdd;
  if constexpr (RowShare<L>::PACK && !ODD)
    return PackRef<A, STREAM, EDGE == kEdgeCut>(m, t, rows, H, RowShare<L>::place());
  else if constexpr (RowShare<L>::PACK)
    return RowRef<A, true, STREAM>(m, static_cast<size_t>(t) * H, H, t < rows);
  else
    return RowRef<A, ODD, STREAM>(m, static_cast<size_t>(t) * H, H);
}

// Sum over the L lanes (8 to 64) of each lane's row, in every one of them, in
// a fixed association.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (L == 64) return wave_sum_f32(v);
  v += __uint_as_float(dpp_u32<kDppXor1>(__float_as_uint(v)));
  v += __uint_as_float(dpp_u32<kDppXor2>(__float_as_uint(v)));
  v += __uint_as_float(dpp_u32<kDppHalfMirror>(__float_as_uint(v)));
  if constexpr (L >= 16) v += __uint_as_float(dpp_u32<kDppMirror>(__float_as_uint(v)));
  if constexpr (L >= 32) v += wave_shfl_xor(v, 16);
  return v;
}

// Sums of one or two values per thread over the threads of a row, in a fixed
// association, the results in every thread.  A workgroup's row (L = 0) goes
// through `slot`, one float (2) per wave in LDS that no other reduction uses
// until the next barrier after this one.
template <int L>
__device__ __forceinline__ float row_sum(float v, float* slot) {
  v = lanes_sum<L == 0 ? 64 : L>(v);
  if constexpr (L == 0) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slot[0];
    for (unsigned i = 1; i < blockDim.x >> 6; ++i) v += slot[i];
  }
  return v;
}

template <int L>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* slot) {
  float2 v = make_float2(lanes_sum<L == 0 ? 64 : L>(a), lanes_sum<L == 0 ? 64 : L>(b));
  if constexpr (L == 0) {
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

// sigmoid(g) for a gradient, which needs G and 1 - G: the smaller of the two,
// e / (1 + e) with e = exp(-|g|), and the sign of g, which says which one it
// is.  One float, and the slope G (1 - G) loses nothing on either side (from
// a rounded G it was 0.05% off at g = 10, 17% at 15 and 0 from 17 on; full
// gates, gradient of 4096 x 2560 bf16 27.4 -> 28.1 us, 16384 x 1024 34.2 ->
// 36.1).  EXACT as in sigmoid().
template <bool EXACT>
__device__ __forceinline__ float sigmoid_tail(float g) {
  const float a = fabsf(g), e = EXACT ? expf(-a) : __builtin_amdgcn_exp2f(-1.44269504088896f * a);
  const float m = e * __builtin_amdgcn_rcpf(1.0f + e);
  // a comparison: copysign's mask took an 81st scalar register, and two
  // workgroups of 1024 threads fit a CU with 80 (gradient of 2048 x 8192
  // float32 41.7 us, 47.2 with the mask)
  return g < 0.f ? -m : m;
}
// G of a tail
__device__ __forceinline__ float tail_sigmoid(float q) {
  return __float_as_int(q) < 0 ? -q : 1.f - q;
}
// G (1 - G)
__device__ __forceinline__ float tail_slope(float q) { return fmaf(-q, q, fabsf(q)); }

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
