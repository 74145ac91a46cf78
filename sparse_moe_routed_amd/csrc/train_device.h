// Device helpers of the training kernels: tiles of two matrices staged through
// LDS and multiplied on the matrix cores, for bf16 and float32 alike.
//
// A product D[m][n] = sum_k M(m, k) N(n, k) is computed in tiles of BM x 128
// outputs by four waves, 2 x 2, each BM/2 x 64.  A stage holds 128 bytes of k
// per row: 64 bf16 or 32 float32.  The N side is MFMA's first operand and the
// M side its second, so a lane of the result (i = lane % 16, q = lane / 16)
// holds values of column-index q and row-index i: with n = 16 q + 4 f + j for
// fragment f it owns 16 neighbouring n of one row m, which it stores itself in
// 16-byte pieces.
//
// Either side comes in one of two forms:
//   rows:    k is contiguous in memory.  LDS holds [row][128 bytes of k].
//   columns: n (or m) is contiguous.  LDS holds [k][128 elements]; bf16 is read
//            back through the transposing LDS read, float32 element by element.
// Stages arrive by buffer loads straight into LDS (no registers): lane l of a
// wave's load writes bytes 16 l .. of 1 KB, so the layout is permuted on the
// source side.  The 16-byte chunk at position p of an LDS row is source chunk
// p ^ key(row), with keys such that the lanes of one LDS read meet distinct
// banks.  What must not be there (rows past the tile, k past the end) is
// loaded from an offset outside the buffer, which leaves zeros in LDS.
#pragma once

#include "moe_device.h"
#include "row_device.h"

namespace moe {

#define MOE_LDS __attribute__((address_space(3)))

constexpr int kStageBytes = 128;            // bytes of k per row and stage
constexpr int kSideBytes = 128 * kStageBytes;
constexpr uint32_t kBufBytes = 0xFFFFFF00u; // no valid offset reaches it
constexpr uint32_t kNowhere = 0xFFFFFFF0u;  // past every buffer: zeros

struct TBf16 {
  typedef uint16_t T;
  typedef RowBf16 Row;
  static constexpr int SZ = 2;
  static constexpr int BK = 64;      // k per stage
  static constexpr int KS = 2;       // MFMA steps per stage
  static __device__ __forceinline__ f32x4_t mma(u32x4_t n, u32x4_t m, f32x4_t c) {
    return mfma_bf16(n, m, c);
  }
  static __device__ __forceinline__ float exp_neg(float g) { return __expf(-g); }
};

struct TF32 {
  typedef float T;
  typedef RowF32 Row;
  static constexpr int SZ = 4;
  static constexpr int BK = 32;
  static constexpr int KS = 2;
  // four steps of v_mfma_f32_16x16x4_f32; element j of lane group q is k = 4 q + j
  static __device__ __forceinline__ f32x4_t mma(u32x4_t n, u32x4_t m, f32x4_t c) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(n[j]), __uint_as_float(m[j]), c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ float exp_neg(float g) { return expf(-g); }
};

typedef __amdgpu_buffer_rsrc_t Rsrc;

__device__ __forceinline__ Rsrc buffer(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(kBufBytes),
                                           0x00020000);
}

__device__ __forceinline__ void load_lds(Rsrc rs, char* lds, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (MOE_LDS void*)lds, 16, static_cast<int>(off), 0, 0, 0);
}

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Keys of the LDS layouts.  Rows form, M side: 16 neighbouring rows of one
// k chunk are read together (two rows per 256-byte line of banks).
__device__ __forceinline__ int key_rows_m(int row) { return (row >> 1) & 7; }
// Rows form, N side (gate and up): rows 8 (i / 4) + i % 4 are read together.
__device__ __forceinline__ int key_rows_n(int row) { return ((row >> 1) & 1) | (((row >> 3) & 3) << 1); }
// Columns form: per k row, bf16 (k rows 8 q + 0..3 together) and float32 (4 q).
template <class E>
__device__ __forceinline__ int key_cols_n(int k) {
  if constexpr (E::SZ == 2) return (k & 3) | (((k >> 3) & 1) << 3);
  return (k >> 2) & 3;
}
template <class E>
__device__ __forceinline__ int key_cols_m(int k) {
  if constexpr (E::SZ == 2) return ((k & 3) << 1) | (((k >> 3) & 1) << 3);
  return ((k >> 2) & 3) << 2;
}

// Load j of wave w covers 1 KB of a side: 8 rows of the rows form (lane l: row
// 8 (4 j + w) + l / 8, position l % 8), or 1024 / (128 SZ) k rows of the
// columns form.
__device__ __forceinline__ int rows_row(int j, int w, int l) { return 8 * (4 * j + w) + (l >> 3); }
template <class E>
__device__ __forceinline__ int cols_k(int j, int w, int l) {
  return E::SZ == 2 ? 4 * (4 * j + w) + (l >> 4) : 2 * (4 * j + w) + (l >> 5);
}
template <class E>
__device__ __forceinline__ int cols_pos(int l) { return l & (E::SZ * 8 - 1); }

// Fragment reads.  ks: MFMA step within the stage.

// rows form, M side: fragment t holds rows m0 + 16 t + i
__device__ __forceinline__ u32x4_t frag_rows_m(const char* s, int m0, int t, int ks, int lane) {
  const int i = lane & 15, q = lane >> 4, row = m0 + 16 * t + i;
  return ld16(s + row * kStageBytes + (((q + 4 * ks) ^ key_rows_m(row)) << 4));
}
// rows form, N side: fragment f of wave wn: gate (f < 2) or up rows 32 wn + 8 (i / 4) + 4 (f % 2) + i % 4
__device__ __forceinline__ u32x4_t frag_rows_n(const char* s, int wn, int f, int ks, int lane) {
  const int i = lane & 15, q = lane >> 4;
  const int row = 64 * (f >> 1) + 32 * wn + 8 * (i >> 2) + 4 * (f & 1) + (i & 3);
  return ld16(s + row * kStageBytes + (((q + 4 * ks) ^ key_rows_n(row)) << 4));
}

// transposing read: lanes 4 c' + r .. see below; gives 4 k of one column
__device__ __forceinline__ u32x2_t lds_transposed(const char* p) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS v4s*)p));
}

// columns form: the fragment's column of result lane i lies in 8-byte chunk
// i / 4 of four (4 bf16 each), element i % 4.  The transposing read takes, in
// each group of 16 lanes, lane 4 r + c's 8 bytes as chunk c of k row r and
// hands lane i the four k of its column.
// N side: column 64 wn + 16 (i / 4) + 4 (f ^ ((i / 4) % 2)) + i % 4: odd lane groups
// take their fragments in swapped order, so that one read meets both halves
// of the 16-byte chunks (unswap() puts the results back).
template <class E>
__device__ __forceinline__ u32x4_t frag_cols_n(const char* s, int wn, int f, int ks, int lane) {
  const int s16 = lane & 15, q = lane >> 4;
  if constexpr (E::SZ == 2) {
    const int c = s16 & 3, k = 32 * ks + 8 * q + (s16 >> 2);
    const int byte = 128 * wn + 32 * c + 8 * (f ^ (c & 1));
    const char* p = s + k * 256 + (((byte >> 4) ^ key_cols_n<E>(k)) << 4) + (byte & 8);
    const u32x2_t lo = lds_transposed(p), hi = lds_transposed(p + 4 * 256);
    return u32x4_t{lo[0], lo[1], hi[0], hi[1]};
  } else {
    const int c = s16 >> 2, k = 16 * ks + 4 * q;
    const int chunk = 16 * wn + 4 * c + (f ^ (c & 1));
    const char* p = s + k * 512 + ((chunk ^ key_cols_n<E>(k)) << 4) + 4 * (s16 & 3);
    u32x4_t v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint32_t*>(p + j * 512);
    return v;
  }
}
// M side: column 64 wm + 16 t + i
template <class E>
__device__ __forceinline__ u32x4_t frag_cols_m(const char* s, int wm, int t, int ks, int lane) {
  const int s16 = lane & 15, q = lane >> 4;
  if constexpr (E::SZ == 2) {
    const int c = s16 & 3, k = 32 * ks + 8 * q + (s16 >> 2);
    const int byte = 128 * wm + 32 * t + 8 * c;
    const char* p = s + k * 256 + (((byte >> 4) ^ key_cols_m<E>(k)) << 4) + (byte & 8);
    const u32x2_t lo = lds_transposed(p), hi = lds_transposed(p + 4 * 256);
    return u32x4_t{lo[0], lo[1], hi[0], hi[1]};
  } else {
    const int k = 16 * ks + 4 * q, chunk = 16 * wm + 4 * t + (s16 >> 2);
    const char* p = s + k * 512 + ((chunk ^ key_cols_m<E>(k)) << 4) + 4 * (s16 & 3);
    u32x4_t v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint32_t*>(p + j * 512);
    return v;
  }
}

// Results of frag_cols_n in the order of n: v[4 f + j] of lane group q is column 16 q + 4 f + j.
__device__ __forceinline__ void unswap(f32x4_t (&a)[4], int lane, float (&v)[16]) {
  const bool odd = (lane >> 4) & 1;
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 * f + j] = odd ? a[f ^ 1][j] : a[f][j];
}

// Two-buffered main loop: stage s + 1 is in flight while stage s is multiplied.
// One barrier a stage: it waits for the own loads (and so, behind it, all
// waves' loads have landed) and says that the other buffer is free again.
template <class Issue, class Compute>
__device__ __forceinline__ void stage_loop(int stages, char* n0, char* m0, char* n1, char* m1,
                                           Issue&& issue, Compute&& compute) {
  if (stages <= 0) return;
  issue(0, n0, m0);
  for (int s = 0;;) {
    __syncthreads();
    if (s + 1 < stages) issue(s + 1, n1, m1);
    compute(n0, m0);
    if (++s >= stages) break;
    __syncthreads();
    if (s + 1 < stages) issue(s + 1, n0, m0);
    compute(n1, m1);
    if (++s >= stages) break;
  }
}

// 16-byte pieces of N elements to and from memory
template <class E, int N>
__device__ __forceinline__ void store_vals(typename E::T* p, const float (&v)[N]) {
  constexpr int V = E::Row::VEC;
#pragma unroll
  for (int c = 0; c < N / V; ++c) {
    float t[V];
#pragma unroll
    for (int e = 0; e < V; ++e) t[e] = v[c * V + e];
    *reinterpret_cast<u32x4_t*>(p + c * V) = E::Row::pack(t);
  }
}
template <class E, int N>
__device__ __forceinline__ void load_vals(const typename E::T* p, float (&v)[N]) {
  constexpr int V = E::Row::VEC;
#pragma unroll
  for (int c = 0; c < N / V; ++c) {
    float t[V];
    E::Row::unpack(ld16(p + c * V), t);
#pragma unroll
    for (int e = 0; e < V; ++e) v[c * V + e] = t[e];
  }
}

// ---- 8-bit checkpoints ----

// Scale byte of 32 elements from the bits of their largest magnitude: the
// smallest b >= 1 with |v| <= 127 * 2^(b - 127) = 1.984375 * 2^(b - 121), at most
// 248 (64 * 2^(249 - 127) would be infinity); 255 where one is not finite.
__device__ __forceinline__ uint32_t scale8(uint32_t top) {
  const int e = static_cast<int>(top >> 23);
  const int b = e - 6 + ((top & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return e == 255 ? 255u : static_cast<uint32_t>(min(max(b, 1), 248));
}
// 2^(127 - b), exact for every b that scale8 gives; a group of scale 255 has codes 0
__device__ __forceinline__ float inverse8(uint32_t b) {
  return b == 255 ? 0.f : __uint_as_float((254u - b) << 23);
}
__device__ __forceinline__ float factor8(uint32_t b) {
  if (b == 255) return __uint_as_float(0x7fc00000u);
  return __uint_as_float(b == 0 ? 0x00400000u : b << 23);
}
// nearest even; the product with a power of two is exact
__device__ __forceinline__ int code8(float v, float inv) {
  return static_cast<int>(inv == 0.f ? 0.f : __builtin_amdgcn_fmed3f(__builtin_rintf(v * inv), -127.f, 127.f));
}
// the codes in the four bytes of w
__device__ __forceinline__ void values8(uint32_t w, float f, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = static_cast<float>(sbfe(w, 8 * i, 8)) * f;
}
__device__ __forceinline__ uint32_t codes8(const float* v, float inv) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= (static_cast<uint32_t>(code8(v[i], inv)) & 0xffu) << (8 * i);
  return w;
}

}  // namespace moe
