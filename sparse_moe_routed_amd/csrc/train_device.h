// Device helpers of the training kernels: tiles of two matrices staged through
// LDS and multiplied on the matrix cores, for bf16 and float32 alike.
//
// A product D[m][n] = sum_k M(m, k) N(n, k) is computed in tiles, each wave 64
// columns (n) of 16, 64 or 128 rows (m).  Few rows: 32 x 128 outputs by four waves (2
// x 2), two stages in LDS (40 KB, four workgroups per CU).  Many rows: 128 x 256 by
// eight waves (2 x 4), three stages (144 KB, one workgroup).  Wide: 256 x 256 by eight
// waves, 32 x 32 matrix instructions, two stages (128 KB).  A stage holds 128 bytes
// of k per row: 64 bf16 or 32 float32.  The N side is MFMA's first operand and the M
// side its second, so a lane of a 16 x 16 result (i = lane % 16, q = lane / 16) holds
// columns 4 q .. 4 q + 3 of a fragment's 16 and row i: after one exchange between
// lanes it stores 8 neighbouring columns (16 bytes of bf16) of its row itself.
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
constexpr int kBlockBytes = 128 * kStageBytes;   // 128 rows, or 128 columns, of a stage
constexpr uint32_t kBufBytes = 0xFFFFFF00u; // no valid offset reaches it
constexpr uint32_t kNowhere = kBufBytes;    // past every buffer: reads zeros, writes nothing

typedef float f32x16_t __attribute__((ext_vector_type(16)));

struct TBf16 {
  typedef uint16_t T;
  typedef RowBf16 Row;
  static constexpr int SZ = 2;
  static constexpr int BK = 64;      // k per stage
  static __device__ __forceinline__ f32x4_t mma(u32x4_t n, u32x4_t m, f32x4_t c) {
    return mfma_bf16(n, m, c);
  }
  // c += ..., in place: the compiler gives an MFMA's result registers of its own,
  // and 128 accumulators twice do not fit.  It does not see a matrix
  // instruction here, so what it would wait for is written out: two states
  // between a vector instruction and an MFMA that reads its result, and, after
  // the last one, mma_done().
  static __device__ __forceinline__ void mma32(u32x4_t n, u32x4_t m, f32x16_t& c) {
    asm("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(c) : "v"(n), "v"(m));
  }
  // exp2 of a rounded product: off by |g| 2^-24 of the value and a few 2^-24, far
  // below the half step 2^-8 of what is made from it
  static __device__ __forceinline__ float exp_neg(float g) { return __expf(-g); }
};

struct TF32 {
  typedef float T;
  typedef RowF32 Row;
  static constexpr int SZ = 4;
  static constexpr int BK = 32;
  // four steps of v_mfma_f32_16x16x4_f32; element j of lane group q is k = 4 q + j
  static __device__ __forceinline__ f32x4_t mma(u32x4_t n, u32x4_t m, f32x4_t c) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(n[j]), __uint_as_float(m[j]), c, 0, 0, 0);
    return c;
  }
  // four steps of v_mfma_f32_32x32x2_f32; element j of lane half h is k = 4 h + j
  static __device__ __forceinline__ void mma32(u32x4_t n, u32x4_t m, f32x16_t& c) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      asm("s_nop 1\n\tv_mfma_f32_32x32x2_f32 %0, %1, %2, %0" : "+v"(c) : "v"(n[j]), "v"(m[j]));
  }
  static __device__ __forceinline__ float exp_neg(float g) { return expf(-g); }
};

// All products of mma32() are done (18 states after the last of 16 passes) and
// may be read.
template <int MF, int NF>
__device__ __forceinline__ void mma_done(f32x16_t (&acc)[MF][NF]) {
  // every product is issued before the waits, every reader stays behind them
#pragma unroll
  for (int t = 0; t < MF; ++t)
#pragma unroll
    for (int f = 0; f < NF; ++f) asm volatile("" : "+v"(acc[t][f]));
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
  for (int t = 0; t < MF; ++t)
#pragma unroll
    for (int f = 0; f < NF; ++f) asm volatile("" : "+v"(acc[t][f]));
}

// A raw buffer as its four words (uniform), for the loads below.
__device__ __forceinline__ u32x4_t buffer(const void* p) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32));
  return u32x4_t{lo, hi & 0xffffu, kBufBytes, 0x00020000u};
}

// 64 lanes x 16 (or 4) bytes from the buffer to LDS, lane l's at lds + 16 l (4 l).
// Written as assembly because the compiler, which knows that such a load
// writes LDS but not where, waits for all of them before the next transposing
// LDS read; here the waits are stage_barrier()'s.  Nothing but LDS is written,
// and the registers are read when the load is issued.  m0 holds the LDS address
// and is declared as overwritten (the warning says that it is not saved, which is
// not wanted; as an operand that the compiler writes it took 0.7% longer: 8192 x
// 2560 x 5120 backward 1384 -> 1394 us).  The five wait states in front are what a
// buffer load needs after the vector unit has written one of its scalar registers.
// stage_barrier()'s counts hold only the memory operations written here: a kernel
// must not spill vector registers.
// ONCE: data that is read about once leaves the caches first (256 tokens, 512 experts of
// 2560 x 640: dh 330 -> 270 us, dx 570 -> 520; where weights are read again, at
// 8192 rows of one expert, it costs: 335 -> 356).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <bool ONCE = false>
__device__ __forceinline__ void load_lds(u32x4_t rs, char* lds, uint32_t off) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>((MOE_LDS char*)lds)));
  if constexpr (ONCE)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, 0 offen nt lds"
                 ::"v"(off), "s"(rs), "s"(at) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 ::"v"(off), "s"(rs), "s"(at) : "memory", "m0");
}
__device__ __forceinline__ void load_lds_word(u32x4_t rs, char* lds, uint32_t off) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>((MOE_LDS char*)lds)));
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tbuffer_load_dword %0, %1, 0 offen lds"
               ::"v"(off), "s"(rs), "s"(at) : "memory", "m0");
}
#pragma clang diagnostic pop

// Rows of expert e within [0, P), whatever the offsets hold.
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int e, int P, int& row0, int& rows) {
  row0 = min(max(offsets[e], 0), P);
  rows = min(max(offsets[e + 1], row0), P) - row0;
}

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Keys of the LDS layouts.  Rows form, M side: 16 neighbouring rows of one
// k chunk are read together (two rows per 256-byte line of banks).
__device__ __forceinline__ int key_rows_m(int row) { return (row >> 1) & 7; }
// Rows form, N side (gate and up): rows 8 (i / 4) + i % 4 are read together.
__device__ __forceinline__ int key_rows_n(int row) { return ((row >> 1) & 1) | (((row >> 3) & 3) << 1); }
// Columns form, per k row: bf16 reads k rows 8 q + 0..3 together, float32 4 q.
template <class E>
__device__ __forceinline__ int key_cols(int k) {
  if constexpr (E::SZ == 2) return ((k & 3) << 1) | (((k >> 3) & 1) << 3);
  return ((k >> 2) & 3) << 2;
}

// Load number i covers 1 KB of a side.  Rows form: rows 8 i .. 8 i + 7 (lane l: row
// 8 i + l / 8, position l % 8).  Columns form, in blocks of 128 columns (16
// loads): 1024 / (128 SZ) k rows of block i / 16.
__device__ __forceinline__ int rows_row(int i, int l) { return 8 * i + (l >> 3); }
template <class E>
__device__ __forceinline__ int cols_k(int i, int l) {
  return E::SZ == 2 ? 4 * (i & 15) + (l >> 4) : 2 * (i & 15) + (l >> 5);
}
template <class E>
__device__ __forceinline__ int cols_pos(int l) { return l & (E::SZ * 8 - 1); }

// Fragment reads.  ks: MFMA step within the stage.

// rows form, M side: fragment t holds rows m0 + 16 t + i
__device__ __forceinline__ u32x4_t frag_rows_m(const char* s, int m0, int t, int ks, int lane) {
  const int i = lane & 15, q = lane >> 4, row = m0 + 16 * t + i;
  return ld16(s + row * kStageBytes + (((q + 4 * ks) ^ key_rows_m(row)) << 4));
}
// rows form, N side: fragment f of wave wn of NW: row 32 wn + 8 (i / 4) + 4 (f % 2) + i % 4 of
// gate (f < 2) or of up, behind the 32 NW rows of gate; a result lane has 8
// neighbouring ones
template <int NW>
__device__ __forceinline__ u32x4_t frag_rows_n(const char* s, int wn, int f, int ks, int lane) {
  const int i = lane & 15, q = lane >> 4;
  const int row = 32 * NW * (f >> 1) + 32 * wn + 8 * (i >> 2) + 4 * (f & 1) + (i & 3);
  return ld16(s + row * kStageBytes + (((q + 4 * ks) ^ key_rows_n(row)) << 4));
}

// transposing read: lanes 4 c' + r .. see below; gives 4 k of one column
__device__ __forceinline__ u32x2_t lds_transposed(const char* p) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS v4s*)p));
}

// columns form: fragment f holds columns 64 half + 16 f + i of a block.  The
// transposing read takes, in each group of 16 lanes, lane 4 r + c's 8 bytes as
// columns 4 c .. 4 c + 3 of k row r and hands lane i the four k of column i.
template <class E>
__device__ __forceinline__ u32x4_t frag_cols(const char* s, int half, int f, int ks, int lane) {
  const int s16 = lane & 15, q = lane >> 4;
  if constexpr (E::SZ == 2) {
    const int c = s16 & 3, k = 32 * ks + 8 * q + (s16 >> 2);
    const int byte = 128 * half + 32 * f + 8 * c;
    const char* p = s + k * 256 + (((byte >> 4) ^ key_cols<E>(k)) << 4) + (byte & 8);
    const u32x2_t lo = lds_transposed(p), hi = lds_transposed(p + 4 * 256);
    return u32x4_t{lo[0], lo[1], hi[0], hi[1]};
  } else {
    const int k = 16 * ks + 4 * q, chunk = 16 * half + 4 * f + (s16 >> 2);
    const char* p = s + k * 512 + ((chunk ^ key_cols<E>(k)) << 4) + 4 * (s16 & 3);
    u32x4_t v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint32_t*>(p + j * 512);
    return v;
  }
}

// Fragments of the 32 x 32 products (16 bf16 or 8 float32 of k a step): lane i =
// lane % 32 holds one index, lane half h = lane / 32 the k.  A result lane (i, h)
// has row i and column indexes 8 g + 4 h + j; index 8 g + 4 h + j is column 16 h + 4 g + j, so
// that it has 16 neighbouring columns.
__device__ __forceinline__ int col_of_index(int i) { return 16 * ((i >> 2) & 1) + 4 * (i >> 3) + (i & 3); }

__device__ __forceinline__ int key32_rows_n(int row) { return ((row >> 1) & 3) | (((row >> 4) & 1) << 2); }
template <class E>
__device__ __forceinline__ int key32_cols(int k) {
  return E::SZ == 2 ? (k & 3) << 2 : ((k >> 2) & 1) << 3;
}
// rows form
__device__ __forceinline__ u32x4_t frag32_rows_m(const char* s, int row0, int ks, int lane) {
  const int row = row0 + (lane & 31);
  return ld16(s + row * kStageBytes + (((2 * ks + (lane >> 5)) ^ key_rows_m(row)) << 4));
}
__device__ __forceinline__ u32x4_t frag32_rows_n(const char* s, int row0, int ks, int lane) {
  const int row = row0 + col_of_index(lane & 31);
  return ld16(s + row * kStageBytes + (((2 * ks + (lane >> 5)) ^ key32_rows_n(row)) << 4));
}
// columns form, columns col0 .. + 31 of a block of 128: in index order (N side) or as they lie (M side)
template <class E, bool N>
__device__ __forceinline__ u32x4_t frag32_cols(const char* s, int col0, int ks, int lane) {
  const int h = lane >> 5;
  if constexpr (E::SZ == 2) {
    const int c = lane & 3, second = (lane >> 4) & 1, k = 16 * ks + 8 * h + ((lane & 15) >> 2);
    // first column of this lane's 8 bytes
    const int col = col0 + (N ? 16 * (c & 1) + 4 * (2 * second + (c >> 1)) : 16 * second + 4 * c);
    const char* p = s + k * 256 + (((col >> 3) ^ key32_cols<E>(k)) << 4) + 2 * (col & 4);
    const u32x2_t lo = lds_transposed(p), hi = lds_transposed(p + 4 * 256);
    return u32x4_t{lo[0], lo[1], hi[0], hi[1]};
  } else {
    const int k = 8 * ks + 4 * h, col = col0 + (N ? col_of_index(lane & 31) : lane & 31);
    const char* p = s + k * 512 + (((col >> 2) ^ key32_cols<E>(k)) << 4) + 4 * (col & 3);
    u32x4_t v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint32_t*>(p + j * 512);
    return v;
  }
}

// A lane's results of a row: fragment f holds columns 16 f + 4 q .. + 3.  Exchanging
// fragments f and f + 1 between lane groups q and q ^ 1 leaves each lane with 8
// neighbouring columns, pair_col(f / 2) .. + 7, of the 32.
__device__ __forceinline__ void swap_pair(float& a, float& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
__device__ __forceinline__ int pair_col(int pair, int lane) {
  const int q = lane >> 4;
  return 32 * pair + 16 * (q & 1) + 8 * (q >> 1);
}
// the 8 columns of fragments 2 pair and 2 pair + 1
__device__ __forceinline__ void pair_vals(const f32x4_t (&a)[4], int pair, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = a[2 * pair][j];
    v[4 + j] = a[2 * pair + 1][j];
    swap_pair(v[j], v[4 + j]);
  }
}

// Lanes 8 .. 15 of each 16 of `a` against lanes 0 .. 7 of `b`.  Where a lane i holds
// a piece of row i, `a` is left with two pieces each of rows 0 .. 7, in lanes i and
// i + 8, and `b` with those of rows 8 .. 15.
__device__ __forceinline__ void swap_rows(u32x4_t& a, u32x4_t& b) {
  constexpr int kRor8 = 0x128;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int x = static_cast<int>(a[j]), y = static_cast<int>(b[j]);
    a[j] = __builtin_amdgcn_update_dpp(x, y, kRor8, 0xF, 0xC, false);
    b[j] = __builtin_amdgcn_update_dpp(y, x, kRor8, 0xF, 0x3, false);
  }
}

// Results a[4] of 16 rows and 64 columns as stores of whole cache lines (128 bytes):
// f(row, column, piece) takes 16 bytes of each lane.
template <class E, class F>
__device__ __forceinline__ void line_pieces(const f32x4_t (&a)[4], int lane, F&& f) {
  const int row = lane & 7, second = (lane >> 3) & 1;
  if constexpr (E::SZ == 2) {
    float v[2][8];
    pair_vals(a, 0, v[0]);
    pair_vals(a, 1, v[1]);
    u32x4_t x = E::Row::pack(v[0]), y = E::Row::pack(v[1]);
    swap_rows(x, y);
    f(row, pair_col(second, lane), x);
    f(row + 8, pair_col(second, lane), y);
  } else {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      u32x4_t x = __builtin_bit_cast(u32x4_t, a[2 * p]), y = __builtin_bit_cast(u32x4_t, a[2 * p + 1]);
      swap_rows(x, y);
      f(row, 32 * p + 16 * second + 4 * (lane >> 4), x);
      f(row + 8, 32 * p + 16 * second + 4 * (lane >> 4), y);
    }
  }
}

// Division by the number of slots (by the round-up method of Granlund and
// Montgomery, "Division by invariant integers using multiplication", 1994): p / k = (t + ((p - t) >> 1)) >> s with t = high word of
// p m, m = floor(2^32 (2^(s + 1) - k) / k) + 1, 2^s < k <= 2^(s + 1), for any 32-bit p.
struct PairDiv {
  uint32_t k, m, s;
  static PairDiv of(int k) {
    PairDiv d{static_cast<uint32_t>(k), 0, 0};
    while ((uint64_t{2} << d.s) < d.k) ++d.s;
    d.m = static_cast<uint32_t>(((uint64_t{1} << 32) * ((uint64_t{2} << d.s) - d.k)) / d.k + 1);
    return d;
  }
  __device__ __forceinline__ uint32_t div(uint32_t p) const {
    if (k == 1) return p;
    const uint32_t t = __umulhi(p, m);
    return (t + ((p - t) >> 1)) >> s;
  }
};

// This wave's loads into LDS but for the `YOUNGER` memory operations issued
// after them are done, and so, behind the barrier, are those of all waves; all
// LDS reads before it are done too.  Memory operations count in order of issue.
template <int YOUNGER>
__device__ __forceinline__ void stage_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(YOUNGER) : "memory");
}

// Keeps instructions on either side apart.
__device__ __forceinline__ void sched_fence() { __builtin_amdgcn_sched_barrier(0); }

// Main loop over a ring of R stages in LDS, KS steps and GROUP loads of a wave
// each.  The fragments of a step are read while the step before it is
// multiplied, so LDS and the matrix cores work at the same time.  The barrier
// of stage s stands before its last step's products: behind it the loads of
// stage s + 1 have landed and all of stage s has been read, so stage s + R goes
// into its place at once.
//   issue(s, stage): starts the loads of stage s;  read(stage, ks, frags);  mma(frags)
template <int R, int KS, int GROUP, class F, class Issue, class Read, class Mma>
__device__ __forceinline__ void ring_loop(int stages, char* ring, int bytes, F& even, F& odd, Issue&& issue,
                                          Read&& read, Mma&& mma) {
  static_assert(KS % 2 == 0, "steps take the fragments in turn");
  if (stages <= 0) return;
#pragma unroll
  for (int s = 0; s < R; ++s)
    if (s < stages) issue(s, ring + s * bytes);
  if (stages >= R)
    stage_barrier<GROUP * (R - 1)>();
  else
    stage_barrier<0>();
  read(ring, 0, even);
  int now = 0;   // offset of stage s
  const auto steps = [&] {   // all but the last one's products
#pragma unroll
    for (int ks = 0; ks + 1 < KS; ++ks) {
      read(ring + now, ks + 1, ks & 1 ? even : odd);
      sched_fence();
      mma(ks & 1 ? odd : even);
      sched_fence();
    }
  };
  for (int s = 0; s + 1 < stages; ++s) {
    steps();
    const int next = now == (R - 1) * bytes ? 0 : now + bytes;
    if (s + R - 1 < stages)
      stage_barrier<GROUP * (R - 2)>();
    else
      stage_barrier<0>();
    if (s + R < stages) issue(s + R, ring + now);
    read(ring + next, 0, even);
    sched_fence();
    mma(odd);
    now = next;
  }
  steps();
  mma(odd);
}

// 16 bytes to an offset of a buffer, nothing to kNowhere; the line leaves the caches
// first.  That pays where all of its 128 bytes are written together: with half lines
// the stores reach 2.5 TB/s and not 5.
__device__ __forceinline__ void store_piece(const void* base, uint32_t off, u32x4_t v) {
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<void*>(base), 0, static_cast<int>(kBufBytes), 0x00020000);
  __builtin_amdgcn_raw_buffer_store_b128(v, rs, static_cast<int>(off), 0, 2);
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
