// The products of the training calls that go over the rows of the experts: the
// gated product that keeps g and u, and the gradient's
//   k_dh:  dh = dy W_down       (sum over H; W_down [H][I] has I contiguous),
//          turned into dg, du and h at once;
//   k_dx:  drows = dg W_gate + du W_up  (sum over I; H contiguous).
// Weights are read as they lie in memory: the transposing LDS read serves the
// sides whose sum index is not contiguous (train_device.h).
//
// What bounds them (the fastest of 12 runs, which is what long rows of calls take too;
// the 5th to 25th call from idle take up to a third more, as a library's products
// do).  Experts of few rows: the weights' bytes (512 experts of 2560 x 640, bf16: 256
// tokens top-10 k_dh 267 us, 6.3 TB/s, k_dx 520 us, 6.5; 4096 tokens k_gate_up_save 760
// to 770, k_dh 465, k_dx 795, 4.3 to 4.9 TB/s with 80 of a tile's 128 rows filled).
// One expert of many rows: the matrix cores (8192 rows of 2560 x 5120: k_gate_up_save
// 395 us, 1090 TFLOP/s, k_dh 326 us with its activations, k_dx 389 + 19).  A handful
// of tiles: the latency of one tile, 7 to 10 us.  One block of tens to hundreds of
// rows: its launches, as a sum that is split is joined by another one (gradient of 53
// rows 3456 x 928 bf16 35 us, of 38 rows 2816 x 1152 float32 60).  Float32 of many rows:
// the matrix cores, on tiles that are filled in part (404 rows an expert in four
// tiles of 128; 640 columns in three slabs of 256).
#pragma once

#include <type_traits>

#include "moe_internal.h"
#include "train_device.h"

namespace moe {

// What the kernels over the rows have in common.
struct RowArgs {
  const int32_t* tiles;   // list of `most` tiles and their number, or NULL: found from offsets
  const int32_t *offsets, *sorted_pair;
  float* part;            // float [parts][P][columns] where the sum is split
  int most, E, H, I, P, parts;
  bool cuts;              // 256 x 256: the last tiles are cut
  PairDiv slots;
};

// Tile, slab of columns and part of the sum of a workgroup; `cut`: parts of this tile's
// sum, `slot` its place among the parts.
struct TileOf {
  int e, row0, rows, slab, part, cut, slot;
};

// Consecutive items run through bands of 8 tiles slab by slab: the tiles of a band
// share a slab's weights where they are of one expert, and a tile's slabs share
// its rows, in an XCD's L2.  `stages` of the whole sum; JOIN: the tiles that were cut.
template <class S, bool JOIN>
__device__ __forceinline__ bool tile_of_block(const RowArgs& a, int slabs, int stages, int block, TileOf& o) {
  constexpr int bm = S::BM;
  int n, row0 = 0, rows = 0, nt = 0, incl = 0;
  if (a.tiles) {
    n = __builtin_amdgcn_readfirstlane(a.tiles[3 * a.most]);
  } else {   // expert = lane
    const int lane = threadIdx.x & 63;
    if (lane < a.E) expert_rows(a.offsets, lane, a.P, row0, rows);
    nt = (rows + bm - 1) / bm;
    incl = wave_incl_scan_i32(nt);
    n = __builtin_amdgcn_readlane(incl, 63);
  }
  slabs *= a.parts;
  const Tail tail(n * slabs, S::WIDE && a.cuts ? stages : 0);
  int item, cut_part = 0;
  o.cut = 1;
  o.slot = 0;
  if constexpr (JOIN) {
    if (block >= tail.rest) return false;
    item = tail.full + block;
    o.slot = block * tail.cut;
    o.cut = tail.cut;
  } else {
    if (!tail.item(block, item, cut_part, o.slot)) return false;
    if (item >= tail.full) o.cut = tail.cut;
  }
  const int band = item / (8 * slabs), rest = item - band * 8 * slabs, wide = min(8, n - 8 * band);
  const int slab = rest / wide, t = 8 * band + rest - slab * wide;
  o.slab = slab / a.parts;
  o.part = S::WIDE ? cut_part : slab - o.slab * a.parts;
  if (!S::WIDE) o.cut = a.parts;
  if (a.tiles) {
    o.e = __builtin_amdgcn_readfirstlane(a.tiles[3 * t]);
    o.row0 = __builtin_amdgcn_readfirstlane(a.tiles[3 * t + 1]);
    o.rows = __builtin_amdgcn_readfirstlane(a.tiles[3 * t + 2]);
  } else {
    o.e = __builtin_ctzll(__ballot(incl > t));
    const int j = t - __builtin_amdgcn_readlane(incl - nt, o.e);
    o.row0 = __builtin_amdgcn_readlane(row0, o.e) + j * bm;
    o.rows = min(__builtin_amdgcn_readlane(rows, o.e) - j * bm, bm);
  }
  return true;
}

// Shapes of a workgroup: MW x NW waves, each 64 columns of MF fragments of rows,
// STAGES in LDS.  PRODUCT: outputs of a matrix instruction, 16 x 16 or 32 x 32.
template <int MW_, int NW_, int MF_, int STAGES_, int PRODUCT, bool ONCE_ = false>
struct Shape {
  static constexpr int MW = MW_, NW = NW_, MF = MF_, STAGES = STAGES_;
  static constexpr bool WIDE = PRODUCT == 32, ONCE = ONCE_;
  static constexpr int NF = 64 / PRODUCT, KS = WIDE ? 4 : 2;       // fragments of columns, steps per stage
  static constexpr int WAVES = MW * NW, THREADS = 64 * WAVES;
  static constexpr int BM = PRODUCT * MF * MW, BN = 64 * NW;
  static constexpr int ML = BM / 8 / WAVES, NL = BN / 8 / WAVES;   // loads of a wave and stage
  static constexpr int NBYTES = BN * kStageBytes, BYTES = NBYTES + BM * kStageBytes;
};
// At 512 experts of 80 rows 128 x 256 is as fast as any shape tried or faster, at 8192
// rows of one expert the gated product takes 500 us with it and 395 with 256 x 256
// (440 with four waves of 128 x 128 in place of eight of 128 x 64).
typedef Shape<2, 2, 1, 2, 16> Few;    // 32 x 128
typedef Shape<2, 4, 4, 3, 16> Many;   // 128 x 256
typedef Shape<2, 2, 1, 2, 16, true> FewOnce;
typedef Shape<2, 4, 4, 3, 16, true> ManyOnce;
typedef Shape<2, 4, 4, 2, 32> Wide;   // 256 x 256

// What the tile products have in common: the waves' places, the layouts, the
// pipeline, and which results a lane has.
template <class E, class S>
struct Tiles {
  struct Frags {
    u32x4_t n[S::NF], m[S::MF];
  };
  typedef typename std::conditional<S::WIDE, f32x16_t, f32x4_t>::type Acc;
  int w, lane, wm, wn;
  Acc acc[S::MF][S::NF] = {};
  __device__ __forceinline__ Tiles() : w(wave_id()), lane(threadIdx.x & 63), wm(w / S::NW), wn(w % S::NW) {}

  static __device__ __forceinline__ int key_n(int row) { return S::WIDE ? key32_rows_n(row) : key_rows_n(row); }
  static __device__ __forceinline__ int key_k(int k) { return S::WIDE ? key32_cols<E>(k) : key_cols<E>(k); }

  // Offsets of the M side's loads in rows form: `at(row)` gives the byte offset
  // of a tile row, rows past the tile are nowhere.
  template <class At>
  __device__ __forceinline__ void rows_m(uint32_t (&off)[S::ML], int rows, At&& at) const {
#pragma unroll
    for (int j = 0; j < S::ML; ++j) {
      const int r = rows_row(j * S::WAVES + w, lane);
      off[j] = r < rows ? at(r) + static_cast<uint32_t>(((lane & 7) ^ key_rows_m(r)) << 4) : kNowhere;
    }
  }
  // Offsets of a side's loads in columns form; columns from `cols` on are
  // nowhere.  krow: the loads' k rows.
  template <int L>
  __device__ __forceinline__ void cols(uint32_t (&off)[L], int (&krow)[L], uint32_t pitch, int cols) const {
#pragma unroll
    for (int j = 0; j < L; ++j) {
      const int i = j * S::WAVES + w, k = cols_k<E>(i, lane);
      const int c = 128 * (i >> 4) + (cols_pos<E>(lane) ^ key_k(k)) * (16 / E::SZ);
      krow[j] = k;
      off[j] = c < cols ? static_cast<uint32_t>(k) * pitch + static_cast<uint32_t>(c * E::SZ) : kNowhere;
    }
  }
  __device__ __forceinline__ void load_n(int j, u32x4_t rs, char* stage, uint32_t off) const {
    load_lds<S::ONCE>(rs, stage + (j * S::WAVES + w) * 1024, off);
  }
  __device__ __forceinline__ void load_m(int j, u32x4_t rs, char* stage, uint32_t off) const {
    load_lds(rs, stage + S::NBYTES + (j * S::WAVES + w) * 1024, off);
  }
  // issue(s, stage), read(stage, ks, frags)
  template <class Issue, class Read>
  __device__ __forceinline__ void run(int stages, char* lds, Issue&& issue, Read&& read) {
    Frags even, odd;
    ring_loop<S::STAGES, S::KS, S::ML + S::NL>(stages, lds, S::BYTES, even, odd, issue, read,
                                               [&](const Frags& f) { mma(f); });
    if constexpr (S::WIDE) mma_done(acc);
  }
  __device__ __forceinline__ void mma(const Frags& f) {
#pragma unroll
    for (int t = 0; t < S::MF; ++t)
#pragma unroll
      for (int i = 0; i < S::NF; ++i) {
        if constexpr (S::WIDE)
          E::mma32(f.n[i], f.m[t], acc[t][i]);
        else
          acc[t][i] = E::mma(f.n[i], f.m[t], acc[t][i]);
      }
  }
  // The sums of a part of a tile that is cut, as the lanes hold them, and all parts' sum.
  __device__ __forceinline__ void store_cut(float* part, int slot) const {
    f32x4_t* p = reinterpret_cast<f32x4_t*>(part + static_cast<size_t>(slot) * (kTailBytes / 4)) + threadIdx.x;
#pragma unroll
    for (int t = 0; t < S::MF; ++t)
#pragma unroll
      for (int i = 0; i < S::NF; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          p[((t * S::NF + i) * 4 + q) * S::THREADS] =
              f32x4_t{acc[t][i][4 * q], acc[t][i][4 * q + 1], acc[t][i][4 * q + 2], acc[t][i][4 * q + 3]};
  }
  __device__ __forceinline__ void add_cuts(const float* part, int slot, int cuts) {
    for (int c = 0; c < cuts; ++c) {
      const f32x4_t* p = reinterpret_cast<const f32x4_t*>(part + static_cast<size_t>(slot + c) * (kTailBytes / 4)) + threadIdx.x;
#pragma unroll
      for (int t = 0; t < S::MF; ++t)
#pragma unroll
        for (int i = 0; i < S::NF; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x4_t v = p[((t * S::NF + i) * 4 + q) * S::THREADS];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[t][i][4 * q + j] += v[j];
          }
    }
  }
  // M side in rows form
  __device__ __forceinline__ void read_m(const char* stage, int ks, Frags& f) const {
    const char* mb = stage + S::NBYTES;
#pragma unroll
    for (int t = 0; t < S::MF; ++t)
      f.m[t] = S::WIDE ? frag32_rows_m(mb, 32 * (S::MF * wm + t), ks, lane)
                       : frag_rows_m(mb, 16 * S::MF * wm, t, ks, lane);
  }
  // N side in rows form: gate and, BN / 2 rows behind it, up
  __device__ __forceinline__ void read_gate_up(const char* stage, int ks, Frags& f) const {
#pragma unroll
    for (int i = 0; i < S::NF; ++i)
      f.n[i] = S::WIDE ? frag32_rows_n(stage, S::BN / 2 * i + 32 * wn, ks, lane)
                       : frag_rows_n<S::NW>(stage, wn, i, ks, lane);
  }
  // N side in columns form
  __device__ __forceinline__ void read_n(const char* stage, int ks, Frags& f) const {
    const char* nb = stage + (wn >> 1) * kBlockBytes;
#pragma unroll
    for (int i = 0; i < S::NF; ++i)
      f.n[i] = S::WIDE ? frag32_cols<E, true>(nb, 64 * (wn & 1) + 32 * i, ks, lane)
                       : frag_cols<E>(nb, wn & 1, i, ks, lane);
  }

  // This lane's results of the tile: rows row(t), t < MF, and of each the 8
  // columns from col(p), p < PAIRS.
  static constexpr int PAIRS = S::WIDE ? 4 : 2;
  __device__ __forceinline__ int row(int t) const {
    return S::WIDE ? 32 * (S::MF * wm + t) + (lane & 31) : 16 * (S::MF * wm + t) + (lane & 15);
  }
  __device__ __forceinline__ int col(int p) const {
    return 64 * wn + (S::WIDE ? 32 * (p >> 1) + 16 * (lane >> 5) + 8 * (p & 1) : pair_col(p, lane));
  }
  __device__ __forceinline__ void vals(int t, int p, float (&v)[8]) const {
    if constexpr (S::WIDE) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = acc[t][p >> 1][8 * (p & 1) + j];
    } else {
      pair_vals(acc[t], p, v);
    }
  }
  // Gated product: COLS neighbouring columns of gate and the same of up, from
  // gate_col(), within 32 that the lanes of `all` share.
  static constexpr int COLS = S::WIDE ? 16 : 8;
  __device__ __forceinline__ int gate_col() const {
    return 32 * wn + (S::WIDE ? 16 * (lane >> 5) : 8 * (lane >> 4));
  }
  __device__ __forceinline__ void gate_up(int t, float (&g)[COLS], float (&u)[COLS]) const {
#pragma unroll
    for (int j = 0; j < COLS; ++j) {
      if constexpr (S::WIDE) {
        g[j] = acc[t][0][j];
        u[j] = acc[t][1][j];
      } else {
        g[j] = acc[t][j >> 2][j & 3];
        u[j] = acc[t][2 + (j >> 2)][j & 3];
      }
    }
  }
  __device__ __forceinline__ uint32_t max_of_32(uint32_t v) const {
    if constexpr (!S::WIDE) v = max(v, wave_shfl_xor(v, 16));
    return max(v, wave_shfl_xor(v, 32));
  }
  __device__ __forceinline__ bool first_of_32() const { return lane < (S::WIDE ? 32 : 16); }
};

// What a kernel leaves: its results in the act type, g and u as 8-bit
// checkpoints, or float32 parts of the sums for a joining kernel.
enum { kOutAct, kOut8, kOutPart };

__device__ __forceinline__ void store_part(float* p, const float (&v)[8]) {
  *reinterpret_cast<f32x4_t*>(p) = f32x4_t{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4_t*>(p + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
}

// ---- gated product ----

struct GateUpOut {
  void *g, *u, *h;
  uint8_t *g_scale, *u_scale;
};

// h, and g and u as they are kept, of C neighbouring columns of a row, given
// what the largest magnitudes' bits of their 32 columns are.
template <class E, int OUT, int C>
__device__ __forceinline__ void store_gate_up(const GateUpOut& o, size_t at, bool first, const float (&g)[C],
                                              const float (&u)[C], uint32_t gtop, uint32_t utop) {
  float h[C];
#pragma unroll
  for (int j = 0; j < C; ++j) h[j] = g[j] / (1.0f + E::exp_neg(g[j])) * u[j];
  store_vals<E>(static_cast<typename E::T*>(o.h) + at, h);
  if constexpr (OUT == kOut8) {
    const uint32_t gs = scale8(gtop), us = scale8(utop);
    const float gi = inverse8(gs), ui = inverse8(us);
#pragma unroll
    for (int j = 0; j < C; j += 8) {
      *reinterpret_cast<u32x2_t*>(static_cast<char*>(o.g) + at + j) = u32x2_t{codes8(g + j, gi), codes8(g + j + 4, gi)};
      *reinterpret_cast<u32x2_t*>(static_cast<char*>(o.u) + at + j) = u32x2_t{codes8(u + j, ui), codes8(u + j + 4, ui)};
    }
    if (first) {
      o.g_scale[at / 32] = static_cast<uint8_t>(gs);
      o.u_scale[at / 32] = static_cast<uint8_t>(us);
    }
  } else {
    store_vals<E>(static_cast<typename E::T*>(o.g) + at, g);
    store_vals<E>(static_cast<typename E::T*>(o.u) + at, u);
  }
}

// The largest magnitude as bits: in the order of magnitude, NaN above infinity.
template <int C>
__device__ __forceinline__ uint32_t top_bits(const float (&v)[C]) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < C; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
  return top;
}

// One tile of BM rows x BN / 2 columns of g and of u.  N side: BN / 2 rows of W_gate
// and the same of W_up, so both factors of h end in the same lane.
template <class E, class S, int OUT, bool JOIN = false>
__global__ __launch_bounds__(S::THREADS, 2) void k_gate_up_save(RowArgs a, const void* __restrict__ x,
                                                                const void* __restrict__ wg,
                                                                const void* __restrict__ wu, GateUpOut o) {
  __shared__ __align__(16) char lds[S::STAGES * S::BYTES];
  constexpr int HALF = S::BN / 2, GL = S::NL / 2;
  const int H = a.H, I = a.I;
  TileOf tl;
  if (!tile_of_block<S, JOIN>(a, (I + HALF - 1) / HALF, H / E::BK, blockIdx.x, tl)) return;
  Tiles<E, S> T;
  const int col0 = tl.slab * HALF, lane = T.lane;
  const size_t wbase = (static_cast<size_t>(tl.e) * I + col0) * H * E::SZ;
  const char* gate = static_cast<const char*>(wg) + wbase;
  const char* up = static_cast<const char*>(wu) + wbase;

  uint32_t moff[S::ML], noff[GL];
  T.rows_m(moff, tl.rows, [&](int r) {
    const int p = min(max(a.sorted_pair[tl.row0 + r], 0), a.P - 1);
    return a.slots.div(static_cast<uint32_t>(p)) * static_cast<uint32_t>(H * E::SZ);
  });
#pragma unroll
  for (int j = 0; j < GL; ++j) {
    const int r = rows_row(j * S::WAVES + T.w, lane);
    noff[j] = col0 + r < I ? static_cast<uint32_t>(r) * (H * E::SZ) +
                                 static_cast<uint32_t>(((lane & 7) ^ T.key_n(r)) << 4)
                           : kNowhere;
  }

  const int stages = H / E::BK, s0 = tl.part * stages / tl.cut;
  const auto products = [&] { T.run(
      (tl.part + 1) * stages / tl.cut - s0, lds,
      [&](int s, char* st) {
        const size_t k = static_cast<size_t>(s0 + s) * kStageBytes;
        const u32x4_t rg = buffer(gate + k), ru = buffer(up + k), rx = buffer(static_cast<const char*>(x) + k);
#pragma unroll
        for (int j = 0; j < GL; ++j) T.load_n(j, rg, st, noff[j]);
#pragma unroll
        for (int j = 0; j < GL; ++j) T.load_n(GL + j, ru, st, noff[j]);
#pragma unroll
        for (int j = 0; j < S::ML; ++j) T.load_m(j, rx, st, moff[j]);
      },
      [&](const char* st, int ks, typename Tiles<E, S>::Frags& f) {
        T.read_gate_up(st, ks, f);
        T.read_m(st, ks, f);
      }); };
  if constexpr (JOIN) {
    T.add_cuts(a.part, tl.slot, tl.cut);
  } else {
    products();
    if constexpr (S::WIDE)
      if (tl.cut > 1) return T.store_cut(a.part, tl.slot);
  }

  constexpr int C = Tiles<E, S>::COLS;
  const int c = col0 + T.gate_col();
#pragma unroll
  for (int t = 0; t < S::MF; ++t) {
    const int r = T.row(t);
    float g[C], u[C];
    T.gate_up(t, g, u);
    uint32_t gtop = 0, utop = 0;
    if constexpr (OUT == kOut8) {
      gtop = T.max_of_32(top_bits(g));
      utop = T.max_of_32(top_bits(u));
    }
    if (r >= tl.rows || c >= I) continue;
    if constexpr (OUT == kOutPart) {
      float* p = a.part + (static_cast<size_t>(tl.part) * a.P + tl.row0 + r) * 2 * I + c;
      store_part(p, g);
      store_part(p + I, u);
    } else {
      store_gate_up<E, OUT>(o, static_cast<size_t>(tl.row0 + r) * I + c, T.first_of_32(), g, u, gtop, utop);
    }
  }
}

// ---- gradient: dh, and dg, du, h from it ----

struct DhArgs {
  const void *g, *u;
  const uint8_t *g_scale, *u_scale;
  void *dg, *du, *h;
};

// dg, du and h of 8 neighbouring columns of a row
template <class E, int OUT>
__device__ __forceinline__ void store_dh(const DhArgs& o, size_t at, const float (&dh)[8]) {
  float g[8], u[8], h[8];
  if constexpr (OUT == kOut8) {
    const u32x2_t gc = *reinterpret_cast<const u32x2_t*>(static_cast<const char*>(o.g) + at);
    const u32x2_t uc = *reinterpret_cast<const u32x2_t*>(static_cast<const char*>(o.u) + at);
    const float gf = factor8(o.g_scale[at / 32]), uf = factor8(o.u_scale[at / 32]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      values8(gc[i], gf, g + 4 * i);
      values8(uc[i], uf, u + 4 * i);
    }
  } else {
    load_vals<E>(static_cast<const typename E::T*>(o.g) + at, g);
    load_vals<E>(static_cast<const typename E::T*>(o.u) + at, u);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float sig = 1.0f / (1.0f + E::exp_neg(g[j])), gs = g[j] * sig;
    h[j] = gs * u[j];
    const float du = dh[j] * gs;
    // dg: the slope, at most 1.1, goes to the larger factor first, so that no product on
    // the way leaves float32's range where the result does not (dh u = 1e42 behind a
    // gate of -60)
    const float slope = sig * (1.0f + g[j] * (1.0f - sig));
    const bool first = fabsf(dh[j]) >= fabsf(u[j]);
    g[j] = (first ? dh[j] : u[j]) * slope * (first ? u[j] : dh[j]);
    u[j] = du;
  }
  store_vals<E>(static_cast<typename E::T*>(o.dg) + at, g);
  store_vals<E>(static_cast<typename E::T*>(o.du) + at, u);
  store_vals<E>(static_cast<typename E::T*>(o.h) + at, h);
}

// dh of one tile of BM rows x BN columns.  Not in the 256 x 256 shape, whose sums
// may be cut at the end: it is slower here.
template <class E, class S, int OUT>
__global__ __launch_bounds__(S::THREADS, 2) void k_dh(RowArgs a, const void* __restrict__ dy,
                                                      const void* __restrict__ wd, DhArgs o) {
  static_assert(!S::WIDE, "no cut tiles here");
  __shared__ __align__(16) char lds[S::STAGES * S::BYTES];
  const int H = a.H, I = a.I;
  TileOf tl;
  if (!tile_of_block<S, false>(a, (I + S::BN - 1) / S::BN, H / E::BK, blockIdx.x, tl)) return;
  Tiles<E, S> T;
  const int col0 = tl.slab * S::BN;
  const char* down = static_cast<const char*>(wd) + (static_cast<size_t>(tl.e) * H * I + col0) * E::SZ;
  const char* rows = static_cast<const char*>(dy) + static_cast<size_t>(tl.row0) * H * E::SZ;

  uint32_t moff[S::ML], noff[S::NL];
  int krow[S::NL];
  T.rows_m(moff, tl.rows, [&](int r) { return static_cast<uint32_t>(r) * static_cast<uint32_t>(H * E::SZ); });
  T.cols(noff, krow, I * E::SZ, I - col0);

  const int stages = H / E::BK, s0 = tl.part * stages / tl.cut;
  T.run(
      (tl.part + 1) * stages / tl.cut - s0, lds,
      [&](int s, char* st) {
        const u32x4_t rn = buffer(down + static_cast<size_t>(s0 + s) * E::BK * I * E::SZ);
        const u32x4_t rm = buffer(rows + static_cast<size_t>(s0 + s) * kStageBytes);
#pragma unroll
        for (int j = 0; j < S::NL; ++j) T.load_n(j, rn, st, noff[j]);
#pragma unroll
        for (int j = 0; j < S::ML; ++j) T.load_m(j, rm, st, moff[j]);
      },
      [&](const char* st, int ks, typename Tiles<E, S>::Frags& f) {
        T.read_n(st, ks, f);
        T.read_m(st, ks, f);
      });

#pragma unroll
  for (int t = 0; t < S::MF; ++t) {
    const int r = T.row(t);
#pragma unroll
    for (int p = 0; p < T.PAIRS; ++p) {
      float dh[8];
      T.vals(t, p, dh);
      const int c = col0 + T.col(p);
      if (r >= tl.rows || c >= I) continue;
      const size_t row = static_cast<size_t>(tl.row0 + r);
      if constexpr (OUT == kOutPart)
        store_part(a.part + (static_cast<size_t>(tl.part) * a.P + row) * I + c, dh);
      else
        store_dh<E, OUT>(o, row * I + c, dh);
    }
  }
}

// ---- gradient: rows ----

// drows of one tile of BM rows x BN columns: the stages run over I twice, dg with
// W_gate, then du with W_up.
template <class E, class S, int OUT, bool JOIN>
__device__ __forceinline__ void dx_tile(const RowArgs& a, const void* __restrict__ dg, const void* __restrict__ du,
                                        const void* __restrict__ wg, const void* __restrict__ wu,
                                        void* __restrict__ drows, char* lds, int block) {
  const int H = a.H, I = a.I;
  TileOf tl;
  if (!tile_of_block<S, JOIN>(a, (H + S::BN - 1) / S::BN, 2 * ((I + E::BK - 1) / E::BK), block, tl)) return;
  Tiles<E, S> T;
  const int col0 = tl.slab * S::BN, half = (I + E::BK - 1) / E::BK;
  const size_t wbase = (static_cast<size_t>(tl.e) * I * H + col0) * E::SZ;
  const size_t rbase = static_cast<size_t>(tl.row0) * I * E::SZ;

  uint32_t moff[S::ML], noff[S::NL];
  int krow[S::NL];
  T.rows_m(moff, tl.rows, [&](int r) { return static_cast<uint32_t>(r) * static_cast<uint32_t>(I * E::SZ); });
  T.cols(noff, krow, H * E::SZ, H - col0);
  // first k of this lane's chunk on the M side, the same for all its loads
  const int mchunk = ((T.lane & 7) ^ key_rows_m(rows_row(T.w, T.lane))) * (16 / E::SZ);

  const int stages = 2 * half, s0 = tl.part * stages / tl.cut;
  const auto products = [&] { T.run(
      (tl.part + 1) * stages / tl.cut - s0, lds,
      [&](int i, char* st) {
        const int s = s0 + i, p = s >= half ? s - half : s, left = I - p * E::BK;   // k left from this stage on
        const char* wt = static_cast<const char*>(s >= half ? wu : wg) + wbase;
        const char* dt = static_cast<const char*>(s >= half ? du : dg) + rbase;
        const u32x4_t rn = buffer(wt + static_cast<size_t>(p) * E::BK * H * E::SZ);
        const u32x4_t rm = buffer(dt + static_cast<size_t>(p) * kStageBytes);
#pragma unroll
        for (int j = 0; j < S::NL; ++j) T.load_n(j, rn, st, krow[j] < left ? noff[j] : kNowhere);
#pragma unroll
        for (int j = 0; j < S::ML; ++j) T.load_m(j, rm, st, mchunk < left ? moff[j] : kNowhere);
      },
      [&](const char* st, int ks, typename Tiles<E, S>::Frags& f) {
        T.read_n(st, ks, f);
        T.read_m(st, ks, f);
      }); };
  if constexpr (JOIN) {
    T.add_cuts(a.part, tl.slot, tl.cut);
  } else {
    products();
    if constexpr (S::WIDE)
      if (tl.cut > 1) return T.store_cut(a.part, tl.slot);
  }

#pragma unroll
  for (int t = 0; t < S::MF; ++t) {
    const int r = T.row(t);
#pragma unroll
    for (int p = 0; p < T.PAIRS; ++p) {
      float v[8];
      T.vals(t, p, v);
      const int c = col0 + T.col(p);
      if (r >= tl.rows || c >= H) continue;
      const size_t row = static_cast<size_t>(tl.row0 + r);
      if constexpr (OUT == kOutPart)
        store_part(a.part + (static_cast<size_t>(tl.part) * a.P + row) * H + c, v);
      else
        store_vals<E>(static_cast<typename E::T*>(drows) + row * H + c, v);
    }
  }
}
template <class E, class S, int OUT, bool JOIN = false>
__global__ __launch_bounds__(S::THREADS, 2) void k_dx(RowArgs a, const void* __restrict__ dg,
                                                      const void* __restrict__ du, const void* __restrict__ wg,
                                                      const void* __restrict__ wu, void* __restrict__ drows) {
  __shared__ __align__(16) char lds[S::STAGES * S::BYTES];
  dx_tile<E, S, OUT, JOIN>(a, dg, du, wg, wu, drows, lds, blockIdx.x);
}

// ---- joining the parts of the sums: 8 columns a thread, parts in order ----

// Row and first column of this thread; false past the experts' rows.
__device__ __forceinline__ bool join_place(const RowArgs& a, int columns, size_t& row, int& c) {
  const int each = columns / 8;
  const size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  row = i / each;
  c = static_cast<int>(i - row * each) * 8;
  return row < static_cast<size_t>(min(max(a.offsets[a.E], 0), a.P));
}

__device__ __forceinline__ void join(const RowArgs& a, size_t row, int columns, int c, float (&v)[8]) {
  const float* p = a.part + row * columns + c;
  const size_t step = static_cast<size_t>(a.P) * columns;
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = p[j];
  for (int i = 1; i < a.parts; ++i) {
    p += step;
    const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(p), hi = *reinterpret_cast<const f32x4_t*>(p + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] += lo[j];
      v[4 + j] += hi[j];
    }
  }
}

template <class E, int OUT>
__global__ __launch_bounds__(256) void k_join_gate_up(RowArgs a, GateUpOut o) {
  size_t row;
  int c;
  // the four threads of 32 columns go together (I is a multiple of 32)
  if (!join_place(a, a.I, row, c)) return;
  float g[8], u[8];
  join(a, row, 2 * a.I, c, g);
  join(a, row, 2 * a.I, a.I + c, u);
  uint32_t gtop = 0, utop = 0;
  if constexpr (OUT == kOut8) {
    gtop = top_bits(g);
    utop = top_bits(u);
    gtop = max(gtop, dpp_u32<kDppXor1>(gtop));
    utop = max(utop, dpp_u32<kDppXor1>(utop));
    gtop = max(gtop, dpp_u32<kDppXor2>(gtop));
    utop = max(utop, dpp_u32<kDppXor2>(utop));
  }
  store_gate_up<E, OUT>(o, row * a.I + c, (threadIdx.x & 3) == 0, g, u, gtop, utop);
}

template <class E, int OUT>
__global__ __launch_bounds__(256) void k_join_dh(RowArgs a, DhArgs o) {
  size_t row;
  int c;
  if (!join_place(a, a.I, row, c)) return;
  float dh[8];
  join(a, row, a.I, c, dh);
  store_dh<E, OUT>(o, row * a.I + c, dh);
}

template <class E>
__global__ __launch_bounds__(256) void k_join_dx(RowArgs a, void* __restrict__ drows) {
  size_t row;
  int c;
  if (!join_place(a, a.H, row, c)) return;
  float v[8];
  join(a, row, a.H, c, v);
  store_vals<E>(static_cast<typename E::T*>(drows) + row * a.H + c, v);
}

// ---- launches ----

template <typename T>
inline T* at_off(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

template <class S>
int tile_grid(const RowArgs& a, int slabs) {
  const int tiles = a.P / S::BM + (a.E < a.P ? a.E : a.P);
  return (tiles * slabs * a.parts + 7) / 8 * 8 + (S::WIDE ? kCus : 0);
}
// Whether the last tiles are cut: the tiles of one expert are known here.
template <class S>
bool cuts_tail(const RowArgs& a, int slabs, int stages) {
  if (!S::WIDE || !Tail::possible(stages)) return false;
  return a.E > 1 || Tail((a.P + S::BM - 1) / S::BM * slabs, stages).cut > 1;
}
inline int join_grid(const RowArgs& a, int columns) {
  return static_cast<int>((static_cast<size_t>(a.P) * columns / 8 + 255) / 256);
}

template <class E, class S>
hipError_t run_gate_up(RowArgs a, const void* x, const moe_experts& ex, const GateUpOut& o, hipStream_t st) {
  const int slabs = (2 * a.I + S::BN - 1) / S::BN, grid = tile_grid<S>(a, slabs);
  a.cuts = cuts_tail<S>(a, slabs, a.H / E::BK);
  const bool q8 = o.g_scale != nullptr;
  if constexpr (!S::WIDE) {
    if (a.parts > 1) {
      k_gate_up_save<E, S, kOutPart><<<grid, S::THREADS, 0, st>>>(a, x, ex.gate, ex.up, o);
      if (const hipError_t e = hipGetLastError()) return e;
      const auto kernel = q8 ? k_join_gate_up<E, kOut8> : k_join_gate_up<E, kOutAct>;
      kernel<<<join_grid(a, a.I), 256, 0, st>>>(a, o);
      return hipGetLastError();
    }
  }
  const auto kernel = q8 ? k_gate_up_save<E, S, kOut8> : k_gate_up_save<E, S, kOutAct>;
  kernel<<<grid, S::THREADS, 0, st>>>(a, x, ex.gate, ex.up, o);
  if constexpr (S::WIDE)
    if (a.cuts) {
      if (const hipError_t e = hipGetLastError()) return e;
      const auto join = q8 ? k_gate_up_save<E, S, kOut8, true> : k_gate_up_save<E, S, kOutAct, true>;
      join<<<kCus / 2, S::THREADS, 0, st>>>(a, x, ex.gate, ex.up, o);
    }
  return hipGetLastError();
}

template <class E, class S>
hipError_t run_dh(const RowArgs& a, const void* dy, const void* down, const DhArgs& o, hipStream_t st) {
  const int grid = tile_grid<S>(a, (a.I + S::BN - 1) / S::BN);
  const bool q8 = o.g_scale != nullptr;
  if (a.parts > 1) {
    k_dh<E, S, kOutPart><<<grid, S::THREADS, 0, st>>>(a, dy, down, o);
    if (const hipError_t e = hipGetLastError()) return e;
    const auto kernel = q8 ? k_join_dh<E, kOut8> : k_join_dh<E, kOutAct>;
    kernel<<<join_grid(a, a.I), 256, 0, st>>>(a, o);
    return hipGetLastError();
  }
  const auto kernel = q8 ? k_dh<E, S, kOut8> : k_dh<E, S, kOutAct>;
  kernel<<<grid, S::THREADS, 0, st>>>(a, dy, down, o);
  return hipGetLastError();
}

template <class E, class S>
hipError_t run_dx(RowArgs a, const DhArgs& d, const moe_experts& ex, void* drows, hipStream_t st) {
  const int slabs = (a.H + S::BN - 1) / S::BN, grid = tile_grid<S>(a, slabs);
  a.cuts = cuts_tail<S>(a, slabs, 2 * ((a.I + E::BK - 1) / E::BK));
  if constexpr (!S::WIDE) {
    if (a.parts > 1) {
      k_dx<E, S, kOutPart><<<grid, S::THREADS, 0, st>>>(a, d.dg, d.du, ex.gate, ex.up, drows);
      if (const hipError_t e = hipGetLastError()) return e;
      k_join_dx<E><<<join_grid(a, a.H), 256, 0, st>>>(a, drows);
      return hipGetLastError();
    }
  }
  k_dx<E, S, kOutAct><<<grid, S::THREADS, 0, st>>>(a, d.dg, d.du, ex.gate, ex.up, drows);
  if constexpr (S::WIDE)
    if (a.cuts) {
      if (const hipError_t e = hipGetLastError()) return e;
      k_dx<E, S, kOutAct, true><<<kCus / 2, S::THREADS, 0, st>>>(a, d.dg, d.du, ex.gate, ex.up, drows);
    }
  return hipGetLastError();
}

}  // namespace moe
