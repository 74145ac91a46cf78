// Training of the routed experts: the gated product that keeps g and u, and
// the gradient of the gated product and the down projection.
//
// With rows r of expert e (token t) the gradient is three kinds of product:
//   k_dh:  dh = dy W_down       (sum over H; W_down [H][I] has I contiguous),
//          turned into dg, du and h at once;
//   k_dx:  drows = dg W_gate + du W_up  (sum over I; H contiguous);
//   k_dw:  dW_gate = dg^T x, dW_up = du^T x, dW_down = dy^T h (sum over the
//          expert's rows; both sides have their output index contiguous).
// Weights are read as they lie in memory: the transposing LDS read serves the
// sides whose sum index is not contiguous (train_device.h).
#include <algorithm>

#include "moe_internal.h"
#include "train_device.h"

namespace moe {

// ---- preparation: tiles, tokens of the rows, x from its checkpoint ----

// Rows of expert e within [0, P), whatever the offsets hold.
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int e, int P, int& row0, int& rows) {
  row0 = min(max(offsets[e], 0), P);
  rows = min(max(offsets[e + 1], row0), P) - row0;
}

// Block 0 writes the tiles in expert order, the others the tokens and x.
__global__ __launch_bounds__(256) void k_train_prep(const int32_t* __restrict__ offsets,
                                                    const int32_t* __restrict__ sorted_pair, int E, int P,
                                                    int k, int bm, int max_tiles,
                                                    int32_t* __restrict__ tiles,
                                                    int32_t* __restrict__ token) {
  if (blockIdx.x > 0) {
    for (int r = (blockIdx.x - 1) * 256 + threadIdx.x; r < P; r += (gridDim.x - 1) * 256)
      token[r] = min(max(sorted_pair[r], 0), P - 1) / k;
    return;
  }
  __shared__ int sums[4];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int n[4], mine = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = threadIdx.x * 4 + i;
    int row0 = 0, rows = 0;
    if (e < E) expert_rows(offsets, e, P, row0, rows);
    n[i] = (rows + bm - 1) / bm;
    mine += n[i];
  }
  const int incl = wave_incl_scan_i32(mine);
  if (lane == 63) sums[w] = incl;
  __syncthreads();
  int at = incl - mine, all = 0;
  for (int i = 0; i < 4; ++i) {
    if (i < w) at += sums[i];
    all += sums[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = threadIdx.x * 4 + i;
    int row0 = 0, rows = 0;
    if (e < E) expert_rows(offsets, e, P, row0, rows);
    for (int t = 0; t < n[i]; ++t, ++at)
      if (at < max_tiles) {
        tiles[3 * at] = e;
        tiles[3 * at + 1] = row0 + t * bm;
        tiles[3 * at + 2] = min(rows - t * bm, bm);
      }
  }
  if (threadIdx.x == 0) tiles[3 * max_tiles] = min(all, max_tiles);
}

struct TileOf {
  int e, row0, rows, slab;
};

// Tile and output slab of this workgroup.  Consecutive items go to one XCD
// (workgroups are dealt to the 8 XCDs in turn), and run through bands of 8
// tiles slab by slab: the tiles of a band share a slab's weights where they are
// of one expert, and a tile's slabs share its rows, in that XCD's L2.
__device__ __forceinline__ bool tile_of_block(const int32_t* __restrict__ tiles, int max_tiles,
                                              int slabs, TileOf& o) {
  const int n = __builtin_amdgcn_readfirstlane(tiles[3 * max_tiles]);
  const int total = n * slabs, per = (total + 7) / 8, s = static_cast<int>(blockIdx.x >> 3);
  const int item = static_cast<int>(blockIdx.x & 7) * per + s;
  if (s >= per || item >= total) return false;
  const int band = item / (8 * slabs), rest = item - band * 8 * slabs, wide = min(8, n - 8 * band);
  o.slab = rest / wide;
  const int t = 8 * band + rest - o.slab * wide;
  o.e = __builtin_amdgcn_readfirstlane(tiles[3 * t]);
  o.row0 = __builtin_amdgcn_readfirstlane(tiles[3 * t + 1]);
  o.rows = __builtin_amdgcn_readfirstlane(tiles[3 * t + 2]);
  return true;
}

// Shapes of a workgroup: MW x NW waves of 16 MF x 64 outputs.
template <int MW_, int NW_, int MF_, int STAGES_>
struct Shape {
  static constexpr int STAGES = STAGES_;   // in LDS
  static constexpr int MW = MW_, NW = NW_, MF = MF_, WAVES = MW * NW, THREADS = 64 * WAVES;
  static constexpr int BM = 16 * MF * MW, BN = 64 * NW;
  static constexpr int ML = BM / 8 / WAVES, NL = BN / 8 / WAVES;   // loads of a wave and stage
  static constexpr int NBYTES = BN * kStageBytes, BYTES = NBYTES + BM * kStageBytes;
};
typedef Shape<2, 2, 1, 2> Few;    // 32 x 128
typedef Shape<2, 4, 4, 3> Many;   // 128 x 256

// What the tile products have in common: the waves' places and the pipeline.
template <class E, class S>
struct Tiles {
  int w, lane, wm, wn;
  __device__ __forceinline__ Tiles() : w(wave_id()), lane(threadIdx.x & 63), wm(w / S::NW), wn(w % S::NW) {}

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
  // Offsets of the N side's loads in columns form; columns from `cols` on are
  // nowhere.  krow: the loads' k rows.
  __device__ __forceinline__ void cols_n(uint32_t (&off)[S::NL], int (&krow)[S::NL], uint32_t pitch, int cols) const {
#pragma unroll
    for (int j = 0; j < S::NL; ++j) {
      const int i = j * S::WAVES + w, k = cols_k<E>(i, lane);
      const int c = 128 * (i >> 4) + (cols_pos<E>(lane) ^ key_cols<E>(k)) * (16 / E::SZ);
      krow[j] = k;
      off[j] = c < cols ? static_cast<uint32_t>(k) * pitch + static_cast<uint32_t>(c * E::SZ) : kNowhere;
    }
  }
  __device__ __forceinline__ void load_n(int j, u32x4_t rs, char* stage, uint32_t off) const {
    load_lds(rs, stage + (j * S::WAVES + w) * 1024, off);
  }
  __device__ __forceinline__ void load_m(int j, u32x4_t rs, char* stage, uint32_t off) const {
    load_lds(rs, stage + S::NBYTES + (j * S::WAVES + w) * 1024, off);
  }
  template <class Issue, class Read>
  __device__ __forceinline__ void run(int stages, char* lds, f32x4_t (&acc)[S::MF][4], Issue&& issue, Read&& read) const {
    Frags<S::MF> even, odd;
    ring_loop<S::STAGES, S::ML + S::NL>(stages, lds, S::BYTES, even, odd, issue, read,
                                        [&](const Frags<S::MF>& f) { mma(f, acc); });
  }
  __device__ __forceinline__ void mma(const Frags<S::MF>& f, f32x4_t (&acc)[S::MF][4]) const {
#pragma unroll
    for (int t = 0; t < S::MF; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = E::mma(f.n[i], f.m[t], acc[t][i]);
  }
  // M side in rows form
  __device__ __forceinline__ void read_m(const char* stage, int ks, Frags<S::MF>& f) const {
#pragma unroll
    for (int t = 0; t < S::MF; ++t) f.m[t] = frag_rows_m(stage + S::NBYTES, 16 * S::MF * wm, t, ks, lane);
  }
  // N side in columns form
  __device__ __forceinline__ void read_n(const char* stage, int ks, Frags<S::MF>& f) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) f.n[i] = frag_cols<E>(stage + (wn >> 1) * kBlockBytes, wn & 1, i, ks, lane);
  }
  // row of the tile whose values this lane holds in fragment t, first column of its 8 of a pair
  __device__ __forceinline__ int row(int t) const { return 16 * S::MF * wm + 16 * t + (lane & 15); }
  __device__ __forceinline__ int col(int pair) const { return 64 * wn + pair_col(pair, lane); }
};

// ---- gated product ----

// One tile of BM rows x BN / 2 columns of g and of u.  N side: BN / 2 rows of W_gate
// and the same of W_up, so both factors of h end in the same lane.
template <class E, class S, bool Q8>
__global__ __launch_bounds__(S::THREADS, 2) void k_gate_up_save(
    const void* __restrict__ x, const void* __restrict__ wg, const void* __restrict__ wu,
    const int32_t* __restrict__ tiles, int max_tiles, const int32_t* __restrict__ token, int H, int I,
    void* __restrict__ g_out, void* __restrict__ u_out, uint8_t* __restrict__ g_scale,
    uint8_t* __restrict__ u_scale, void* __restrict__ h_out) {
  __shared__ __align__(16) char lds[S::STAGES * S::BYTES];
  constexpr int HALF = S::BN / 2, GL = S::NL / 2;
  TileOf tl;
  if (!tile_of_block(tiles, max_tiles, (I + HALF - 1) / HALF, tl)) return;
  const Tiles<E, S> T;
  const int col0 = tl.slab * HALF, lane = T.lane;
  const size_t wbase = (static_cast<size_t>(tl.e) * I + col0) * H * E::SZ;
  const char* gate = static_cast<const char*>(wg) + wbase;
  const char* up = static_cast<const char*>(wu) + wbase;

  uint32_t moff[S::ML], noff[GL];
  T.rows_m(moff, tl.rows, [&](int r) {
    return static_cast<uint32_t>(token[tl.row0 + r]) * static_cast<uint32_t>(H * E::SZ);
  });
#pragma unroll
  for (int j = 0; j < GL; ++j) {
    const int r = rows_row(j * S::WAVES + T.w, lane);
    noff[j] = col0 + r < I ? static_cast<uint32_t>(r) * (H * E::SZ) +
                                 static_cast<uint32_t>(((lane & 7) ^ key_rows_n(r)) << 4)
                           : kNowhere;
  }

  f32x4_t acc[S::MF][4] = {};
  T.run(
      H / E::BK, lds, acc,
      [&](int s, char* st) {
        const size_t k = static_cast<size_t>(s) * kStageBytes;
        const u32x4_t rg = buffer(gate + k), ru = buffer(up + k), rx = buffer(static_cast<const char*>(x) + k);
#pragma unroll
        for (int j = 0; j < GL; ++j) T.load_n(j, rg, st, noff[j]);
#pragma unroll
        for (int j = 0; j < GL; ++j) T.load_n(GL + j, ru, st, noff[j]);
#pragma unroll
        for (int j = 0; j < S::ML; ++j) T.load_m(j, rx, st, moff[j]);
      },
      [&](const char* st, int ks, Frags<S::MF>& f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f.n[i] = frag_rows_n<S::NW>(st, T.wn, i, ks, lane);
        T.read_m(st, ks, f);
      });

  // this lane: columns c .. c + 7 of a row
  const int q = lane >> 4, c = col0 + 32 * T.wn + 8 * q;
#pragma unroll
  for (int t = 0; t < S::MF; ++t) {
    const int r = T.row(t);
    float g[8], u[8], h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[j] = acc[t][j >> 2][j & 3];
      u[j] = acc[t][2 + (j >> 2)][j & 3];
      h[j] = g[j] / (1.0f + E::exp_neg(g[j])) * u[j];
    }
    uint32_t gs = 0, us = 0;
    if constexpr (Q8) {
      // the largest magnitude as bits: in the order of magnitude, NaN above infinity
      uint32_t gb = 0, ub = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        gb = max(gb, __float_as_uint(g[j]) & 0x7fffffffu);
        ub = max(ub, __float_as_uint(u[j]) & 0x7fffffffu);
      }
      // the group's other 24 columns are with lane groups q ^ 1, q ^ 2, q ^ 3
      gb = max(gb, wave_shfl_xor(gb, 16));
      ub = max(ub, wave_shfl_xor(ub, 16));
      gs = scale8(max(gb, wave_shfl_xor(gb, 32)));
      us = scale8(max(ub, wave_shfl_xor(ub, 32)));
    }
    if (r >= tl.rows || c >= I) continue;
    const size_t at = static_cast<size_t>(tl.row0 + r) * I + c;
    store_vals<E>(static_cast<typename E::T*>(h_out) + at, h);
    if constexpr (Q8) {
      const float gi = inverse8(gs), ui = inverse8(us);
      *reinterpret_cast<u32x2_t*>(static_cast<char*>(g_out) + at) = u32x2_t{codes8(g, gi), codes8(g + 4, gi)};
      *reinterpret_cast<u32x2_t*>(static_cast<char*>(u_out) + at) = u32x2_t{codes8(u, ui), codes8(u + 4, ui)};
      if (q == 0) {
        g_scale[at / 32] = static_cast<uint8_t>(gs);
        u_scale[at / 32] = static_cast<uint8_t>(us);
      }
    } else {
      store_vals<E>(static_cast<typename E::T*>(g_out) + at, g);
      store_vals<E>(static_cast<typename E::T*>(u_out) + at, u);
    }
  }
}

// ---- gradient: dh, and dg, du, h from it ----

// dh of one tile of BM rows x BN columns.
template <class E, class S, bool Q8>
__global__ __launch_bounds__(S::THREADS, 2) void k_dh(
    const void* __restrict__ dy, const void* __restrict__ wd, const int32_t* __restrict__ tiles,
    int max_tiles, int H, int I, const void* __restrict__ g_in, const void* __restrict__ u_in,
    const uint8_t* __restrict__ g_scale, const uint8_t* __restrict__ u_scale, void* __restrict__ dg_out,
    void* __restrict__ du_out, void* __restrict__ h_out) {
  __shared__ __align__(16) char lds[S::STAGES * S::BYTES];
  TileOf tl;
  if (!tile_of_block(tiles, max_tiles, (I + S::BN - 1) / S::BN, tl)) return;
  const Tiles<E, S> T;
  const int col0 = tl.slab * S::BN;
  const char* down = static_cast<const char*>(wd) + (static_cast<size_t>(tl.e) * H * I + col0) * E::SZ;
  const char* rows = static_cast<const char*>(dy) + static_cast<size_t>(tl.row0) * H * E::SZ;

  uint32_t moff[S::ML], noff[S::NL];
  int krow[S::NL];
  T.rows_m(moff, tl.rows, [&](int r) { return static_cast<uint32_t>(r) * static_cast<uint32_t>(H * E::SZ); });
  T.cols_n(noff, krow, I * E::SZ, I - col0);

  f32x4_t acc[S::MF][4] = {};
  T.run(
      H / E::BK, lds, acc,
      [&](int s, char* st) {
        const u32x4_t rn = buffer(down + static_cast<size_t>(s) * E::BK * I * E::SZ);
        const u32x4_t rm = buffer(rows + static_cast<size_t>(s) * kStageBytes);
#pragma unroll
        for (int j = 0; j < S::NL; ++j) T.load_n(j, rn, st, noff[j]);
#pragma unroll
        for (int j = 0; j < S::ML; ++j) T.load_m(j, rm, st, moff[j]);
      },
      [&](const char* st, int ks, Frags<S::MF>& f) {
        T.read_n(st, ks, f);
        T.read_m(st, ks, f);
      });

#pragma unroll
  for (int t = 0; t < S::MF; ++t) {
    const int r = T.row(t);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      float dh[8], g[8], u[8], h[8];
      pair_vals(acc[t], p, dh);
      const int c = col0 + T.col(p);
      if (r >= tl.rows || c >= I) continue;
      const size_t at = static_cast<size_t>(tl.row0 + r) * I + c;
      if constexpr (Q8) {
        const u32x2_t gc = *reinterpret_cast<const u32x2_t*>(static_cast<const char*>(g_in) + at);
        const u32x2_t uc = *reinterpret_cast<const u32x2_t*>(static_cast<const char*>(u_in) + at);
        const float gf = factor8(g_scale[at / 32]), uf = factor8(u_scale[at / 32]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          values8(gc[i], gf, g + 4 * i);
          values8(uc[i], uf, u + 4 * i);
        }
      } else {
        load_vals<E>(static_cast<const typename E::T*>(g_in) + at, g);
        load_vals<E>(static_cast<const typename E::T*>(u_in) + at, u);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float sig = 1.0f / (1.0f + E::exp_neg(g[j])), gs = g[j] * sig;
        h[j] = gs * u[j];
        const float du = dh[j] * gs;
        g[j] = dh[j] * u[j] * sig * (1.0f + g[j] * (1.0f - sig));   // dg
        u[j] = du;
      }
      store_vals<E>(static_cast<typename E::T*>(dg_out) + at, g);
      store_vals<E>(static_cast<typename E::T*>(du_out) + at, u);
      store_vals<E>(static_cast<typename E::T*>(h_out) + at, h);
    }
  }
}

// ---- gradient: rows ----

// drows of one tile of BM rows x BN columns: the stages run over I twice, dg with
// W_gate, then du with W_up.
template <class E, class S>
__global__ __launch_bounds__(S::THREADS, 2) void k_dx(const void* __restrict__ dg, const void* __restrict__ du,
                                                      const void* __restrict__ wg, const void* __restrict__ wu,
                                                      const int32_t* __restrict__ tiles, int max_tiles, int H,
                                                      int I, void* __restrict__ drows) {
  __shared__ __align__(16) char lds[S::STAGES * S::BYTES];
  TileOf tl;
  if (!tile_of_block(tiles, max_tiles, (H + S::BN - 1) / S::BN, tl)) return;
  const Tiles<E, S> T;
  const int col0 = tl.slab * S::BN, half = (I + E::BK - 1) / E::BK;
  const size_t wbase = (static_cast<size_t>(tl.e) * I * H + col0) * E::SZ;
  const size_t rbase = static_cast<size_t>(tl.row0) * I * E::SZ;

  uint32_t moff[S::ML], noff[S::NL];
  int krow[S::NL];
  T.rows_m(moff, tl.rows, [&](int r) { return static_cast<uint32_t>(r) * static_cast<uint32_t>(I * E::SZ); });
  T.cols_n(noff, krow, H * E::SZ, H - col0);
  // first k of this lane's chunk on the M side, the same for all its loads
  const int mchunk = ((T.lane & 7) ^ key_rows_m(rows_row(T.w, T.lane))) * (16 / E::SZ);

  f32x4_t acc[S::MF][4] = {};
  T.run(
      2 * half, lds, acc,
      [&](int s, char* st) {
        const int p = s >= half ? s - half : s, left = I - p * E::BK;   // k left from this stage on
        const char* wt = static_cast<const char*>(s >= half ? wu : wg) + wbase;
        const char* dt = static_cast<const char*>(s >= half ? du : dg) + rbase;
        const u32x4_t rn = buffer(wt + static_cast<size_t>(p) * E::BK * H * E::SZ);
        const u32x4_t rm = buffer(dt + static_cast<size_t>(p) * kStageBytes);
#pragma unroll
        for (int j = 0; j < S::NL; ++j) T.load_n(j, rn, st, krow[j] < left ? noff[j] : kNowhere);
#pragma unroll
        for (int j = 0; j < S::ML; ++j) T.load_m(j, rm, st, mchunk < left ? moff[j] : kNowhere);
      },
      [&](const char* st, int ks, Frags<S::MF>& f) {
        T.read_n(st, ks, f);
        T.read_m(st, ks, f);
      });

#pragma unroll
  for (int t = 0; t < S::MF; ++t) {
    const int r = T.row(t);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      float v[8];
      pair_vals(acc[t], p, v);
      const int c = col0 + T.col(p);
      if (r < tl.rows && c < H)
        store_vals<E>(static_cast<typename E::T*>(drows) + static_cast<size_t>(tl.row0 + r) * H + c, v);
    }
  }
}

// ---- gradient: weights ----

struct DwArgs {
  const void *dg, *du, *h, *dy, *x;
  void *dgate, *dup, *ddown;
  const int32_t *offsets, *token;
  int E, H, I, P;
  int strip;   // neighbouring tiles of a workgroup
  int unit;    // neighbouring strips on one XCD
};

// A strip of 128 x 128 tiles of a weight gradient, side by side in n, by four
// waves (64 x 64 each, two workgroups per CU).  M side: dg, du [row][I] or dy
// [row][H]; N side: x of the rows' tokens [token][H], or h [row][I].  Both are
// in columns form, with the expert's rows as k.
//
// An expert of at most two stages of rows keeps its M side in registers for the
// whole strip, and only the N side runs through a ring (three stages ahead); with more rows
// both sides run through a ring of two.  Either way the stages of all tiles are
// one pipeline, so the next loads are on their way while a tile is stored.
template <class E>
struct DwStrip {
  typedef Shape<2, 2, 4, 2> S;
  static constexpr int LOADS = 4;                     // of a wave, side and stage
  static constexpr int KR = E::SZ == 2 ? 4 : 2;       // k rows of a load
  static constexpr int TOKEN_BYTES = 256;             // of a wave and stage
  static constexpr int LDS = 4 * kBlockBytes + 4 * S::WAVES * TOKEN_BYTES;
  static constexpr int STORES = 4 * 16 * E::SZ / 16;  // of a thread and tile

  const DwArgs& a;
  char* lds;
  Tiles<E, S> T;
  const char *mside, *nside;   // first row of the expert
  char* out;                   // first row of the strip
  bool gather;
  int mcols, ncols, m0, nt0, tiles, row0, rows, stages;
  int krow[LOADS], chunk[LOADS];   // k row and column of this lane's 16 bytes of load j
  u32x4_t token_rs;
  char* token_lds;
  int token_row;
  int lt = 0, ls = 0, ln = 0;   // tile, stage and number of the next loads
  f32x4_t acc[4][4] = {};

  __device__ __forceinline__ DwStrip(const DwArgs& args, char* shared) : a(args), lds(shared) {}

  __device__ __forceinline__ void init(int e, int which, int mt, int first, int count) {
    const bool down = which == 2;
    gather = !down;
    mcols = down ? a.H : a.I;
    ncols = down ? a.I : a.H;
    m0 = mt * 128;
    nt0 = first;
    tiles = count;
    row0 = rows = 0;
    if (a.P > 0) expert_rows(a.offsets, e, a.P, row0, rows);
    row0 = __builtin_amdgcn_readfirstlane(row0);
    rows = __builtin_amdgcn_readfirstlane(rows);
    stages = (rows + E::BK - 1) / E::BK;
    mside = static_cast<const char*>(down ? a.dy : which ? a.du : a.dg) +
            (static_cast<size_t>(row0) * mcols + m0) * E::SZ;
    nside = down ? static_cast<const char*>(a.h) + static_cast<size_t>(row0) * a.I * E::SZ
                 : static_cast<const char*>(a.x);
    out = static_cast<char*>(down ? a.ddown : which ? a.dup : a.dgate) +
          (static_cast<size_t>(e) * a.I * a.H + static_cast<size_t>(m0) * ncols) * E::SZ;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      krow[j] = cols_k<E>(j * S::WAVES + T.w, T.lane);
      chunk[j] = (cols_pos<E>(T.lane) ^ key_cols<E>(krow[j])) * (16 / E::SZ);
    }
    // The gathered rows' tokens go through LDS too; every wave loads those of its
    // own k rows (lane 8 j + i: row i of load j).  Those of loads n are requested
    // with loads n - 3: loads n are issued when loads n - 3 (few rows) or later
    // ones (many rows) are known to have landed.
    token_rs = buffer(a.token + row0);
    token_lds = lds + 4 * kBlockBytes + T.w * TOKEN_BYTES;
    token_row = cols_k<E>(((T.lane >> 3) & 3) * S::WAVES + T.w, 0) + (T.lane & (KR - 1));
  }

  __device__ __forceinline__ void store_tile(int nt) {
    const char* tile = out + static_cast<size_t>(nt) * 128 * E::SZ;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int r = T.row(t);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        float v[8];
        pair_vals(acc[t], p, v);
        const int c = T.col(p);
        store_vals<E>(tile, nt * 128 + c < ncols && m0 + r < mcols ? static_cast<uint32_t>(r * ncols + c) * E::SZ : kNowhere, v);
      }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int f = 0; f < 4; ++f) acc[t][f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }

  __device__ __forceinline__ void load_tokens(int s, int slot) const {
    load_lds_word(token_rs, token_lds + (slot & 3) * (S::WAVES * TOKEN_BYTES),
                  static_cast<uint32_t>(min(s * E::BK + token_row, rows - 1)) * 4);
  }
  __device__ __forceinline__ int after(int s) const { return s + 1 == stages ? 0 : s + 1; }

  __device__ __forceinline__ void issue_m(int s, char* st) const {
    const int left = rows - s * E::BK;
    const u32x4_t rm = buffer(mside + static_cast<size_t>(s) * E::BK * mcols * E::SZ);
#pragma unroll
    for (int j = 0; j < LOADS; ++j)
      load_lds(rm, st + (j * S::WAVES + T.w) * 1024,
               krow[j] < left && m0 + chunk[j] < mcols
                   ? static_cast<uint32_t>(krow[j] * mcols + chunk[j]) * E::SZ
                   : kNowhere);
  }
  // the next N loads, into `st`, and the tokens of those three further on
  __device__ __forceinline__ void issue_n(char* st) {
    const uint32_t* tok = reinterpret_cast<const uint32_t*>(token_lds + (ln & 3) * (S::WAVES * TOKEN_BYTES));
    const int left = rows - ls * E::BK, n0 = (nt0 + lt) * 128;
    const u32x4_t rn = buffer(nside + (gather ? 0 : static_cast<size_t>(ls) * E::BK * a.I * E::SZ) +
                              static_cast<size_t>(n0) * E::SZ);
    uint32_t off[LOADS];
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const uint32_t token = tok[8 * j + (krow[j] & (KR - 1))];
      const uint32_t row = gather ? token : static_cast<uint32_t>(krow[j]);
      off[j] = krow[j] < left && n0 + chunk[j] < ncols
                   ? row * static_cast<uint32_t>(ncols * E::SZ) + static_cast<uint32_t>(chunk[j] * E::SZ)
                   : kNowhere;
    }
    load_tokens(after(after(after(ls))), ln + 3);
#pragma unroll
    for (int j = 0; j < LOADS; ++j) load_lds(rn, st + (j * S::WAVES + T.w) * 1024, off[j]);
    ++ln;
    if (++ls == stages) {
      ls = 0;
      ++lt;
    }
  }
  __device__ __forceinline__ void first_tokens() const {
    load_tokens(0, 0);
    load_tokens(after(0), 1);
    load_tokens(after(after(0)), 2);
    stage_barrier<0>();
  }

  __device__ __forceinline__ void read_n(const char* st, int ks, u32x4_t (&n)[4]) const {
#pragma unroll
    for (int f = 0; f < 4; ++f) n[f] = frag_cols<E>(st, T.wn, f, ks, T.lane);
  }
  __device__ __forceinline__ void read_m(const char* st, int ks, u32x4_t (&m)[4]) const {
#pragma unroll
    for (int t = 0; t < 4; ++t) m[t] = frag_cols<E>(st, T.wm, t, ks, T.lane);
  }
  __device__ __forceinline__ void mma(const u32x4_t (&n)[4], const u32x4_t (&m)[4]) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int f = 0; f < 4; ++f) acc[t][f] = E::mma(n[f], m[t], acc[t][f]);
  }

  // at most two stages of rows
  __device__ __forceinline__ void run_few() {
    u32x4_t m[2][2][4];   // stage, step
    first_tokens();
    issue_m(0, lds);
    if (stages > 1) issue_m(1, lds + kBlockBytes);
    stage_barrier<0>();
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (s < stages) {
        read_m(lds + s * kBlockBytes, 0, m[s][0]);
        read_m(lds + s * kBlockBytes, 1, m[s][1]);
      }
    stage_barrier<0>();   // all waves have read
    constexpr int GROUP = LOADS + 1;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (lt < tiles) issue_n(lds + i * kBlockBytes);
    int slot = 0;
    for (int t = 0; t < tiles; ++t) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (s >= stages) break;
        // This stage's loads are done.  Younger are those of the two after it and the stores
        // since the third stage before it: those of three tiles of one stage, of one or two of two.
        const int stores = stages == 1 ? t : min(t, 1);
        if (lt == tiles || stores == 0)
          lt == tiles ? stage_barrier<0>() : stage_barrier<2 * GROUP>();
        else if (stores < 3)
          stage_barrier<2 * GROUP + STORES>();
        else
          stage_barrier<2 * GROUP + 3 * STORES>();
        // all waves have read the stage before it
        if (lt < tiles) issue_n(lds + ((slot + 3) & 3) * kBlockBytes);
        const char* st = lds + slot * kBlockBytes;
        u32x4_t n0[4], n1[4];
        read_n(st, 0, n0);
        read_n(st, 1, n1);
        mma(n0, m[s][0]);
        mma(n1, m[s][1]);
        slot = (slot + 1) & 3;
      }
      store_tile(nt0 + t);
    }
  }

  __device__ __forceinline__ void run_many() {
    constexpr int GROUP = 2 * LOADS + 1;
    const auto issue = [&](char* st) {
      issue_m(ls, st + kBlockBytes);
      issue_n(st);
    };
    first_tokens();
    issue(lds);
    if (lt < tiles) issue(lds + 2 * kBlockBytes);
    if (ln == 2)
      stage_barrier<GROUP>();
    else
      stage_barrier<0>();
    u32x4_t n[2][4], m[2][4];   // step
    read_n(lds, 0, n[0]);
    read_m(lds + kBlockBytes, 0, m[0]);
    int now = 0, s = 0;
    bool stored = false;
    for (int nt = nt0, left = tiles * stages;; --left) {
      read_n(lds + now, 1, n[1]);
      read_m(lds + now + kBlockBytes, 1, m[1]);
      sched_fence();
      mma(n[0], m[0]);
      if (left == 1) break;
      const int next = now ^ (2 * kBlockBytes);
      sched_fence();
      if (stored)
        stage_barrier<STORES>();
      else
        stage_barrier<0>();
      if (lt < tiles) issue(lds + now);
      read_n(lds + next, 0, n[0]);
      read_m(lds + next + kBlockBytes, 0, m[0]);
      sched_fence();
      mma(n[1], m[1]);
      now = next;
      stored = ++s == stages;
      if (stored) {
        store_tile(nt++);
        s = 0;
      }
    }
    mma(n[1], m[1]);
    store_tile(nt0 + tiles - 1);
  }
};

template <class E>
__global__ __launch_bounds__(256, 2) void k_dw(DwArgs a) {
  __shared__ __align__(16) char lds[DwStrip<E>::LDS];
  const int it = (a.I + 127) / 128, ht = a.H / 128;
  const int wide = it * ((ht + a.strip - 1) / a.strip), tall = ht * ((it + a.strip - 1) / a.strip);
  const int each = 2 * wide + tall;
  // strips are dealt to the XCDs in units (workgroups in turn)
  const int turn = static_cast<int>(blockIdx.x >> 3), unit = turn / a.unit;
  const int item = (unit * 8 + static_cast<int>(blockIdx.x & 7)) * a.unit + turn - unit * a.unit;
  if (item >= each * a.E) return;
  const int e = item / each, in_e = item - e * each;
  const int which = in_e < wide ? 0 : in_e < 2 * wide ? 1 : 2, ntiles = which == 2 ? it : ht;
  const int strips = (ntiles + a.strip - 1) / a.strip, b = in_e - which * wide;
  const int mt = b / strips, nt0 = (b - mt * strips) * a.strip;
  DwStrip<E> s(a, lds);
  s.init(e, which, mt, nt0, min(a.strip, ntiles - nt0));
  if (s.rows == 0) {
    for (int t = 0; t < s.tiles; ++t) s.store_tile(nt0 + t);
  } else if (s.stages <= 2) {
    s.run_few();
  } else {
    s.run_many();
  }
}

// ---- launches ----

constexpr int kMaxStrip = 20;

template <typename T>
static T* at_off(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

static hipError_t launch_prep(const moe_shape& s, const TrainPlan& pl, const moe_perm& pm, void* ws,
                              hipStream_t st) {
  const int P = s.T * s.top_k;
  const int grid = 1 + static_cast<int>((static_cast<size_t>(P) + 1023) / 1024);
  k_train_prep<<<grid, 256, 0, st>>>(pm.offsets, pm.sorted_pair, s.E, P, s.top_k, pl.bm, pl.max_tiles,
                                     at_off<int32_t>(ws, pl.tiles_off), at_off<int32_t>(ws, pl.token_off));
  return hipGetLastError();
}

static int tile_grid(const TrainPlan& pl, int slabs) { return (pl.max_tiles * slabs + 7) / 8 * 8; }

template <class E, class S, bool Q8>
static void run_gate_up(const moe_shape& s, const TrainPlan& pl, const void* x, const moe_experts& ex,
                        const moe_saved& sv, void* h, void* ws, hipStream_t st) {
  k_gate_up_save<E, S, Q8><<<tile_grid(pl, (2 * s.I + S::BN - 1) / S::BN), S::THREADS, 0, st>>>(
      x, ex.gate, ex.up, at_off<int32_t>(ws, pl.tiles_off), pl.max_tiles, at_off<int32_t>(ws, pl.token_off),
      s.H, s.I, sv.g, sv.u, sv.g_scale, sv.u_scale, h);
}

template <class E, class S>
static void run_gate_up(const moe_shape& s, const TrainPlan& pl, const void* x, const moe_experts& ex,
                        const moe_saved& sv, void* h, void* ws, hipStream_t st) {
  sv.g_scale ? run_gate_up<E, S, true>(s, pl, x, ex, sv, h, ws, st) : run_gate_up<E, S, false>(s, pl, x, ex, sv, h, ws, st);
}

template <class E>
static void run_gate_up(const moe_shape& s, const TrainPlan& pl, const void* x, const moe_experts& ex,
                        const moe_saved& sv, void* h, void* ws, hipStream_t st) {
  pl.bm == Few::BM ? run_gate_up<E, Few>(s, pl, x, ex, sv, h, ws, st) : run_gate_up<E, Many>(s, pl, x, ex, sv, h, ws, st);
}

hipError_t launch_gate_up_save(const moe_shape& s, const TrainPlan& pl, const void* x,
                               const moe_experts& ex, const moe_perm& pm, const moe_saved& sv,
                               void* h, void* ws, hipStream_t st) {
  if (const hipError_t e = launch_prep(s, pl, pm, ws, st)) return e;
  if (s.act == MOE_DT_BF16)
    run_gate_up<TBf16>(s, pl, x, ex, sv, h, ws, st);
  else
    run_gate_up<TF32>(s, pl, x, ex, sv, h, ws, st);
  return hipGetLastError();
}

template <class E, class S>
static hipError_t run_rows(const moe_shape& s, const TrainPlan& pl, const void* dy, const moe_saved& sv,
                           const moe_experts& ex, void* drows, void* ws, hipStream_t st) {
  const int32_t* tiles = at_off<int32_t>(ws, pl.tiles_off);
  void *dg = at_off<char>(ws, pl.dg_off), *du = at_off<char>(ws, pl.du_off), *h = at_off<char>(ws, pl.h_off);
  const int grid = tile_grid(pl, (s.I + S::BN - 1) / S::BN);
  if (sv.g_scale)
    k_dh<E, S, true><<<grid, S::THREADS, 0, st>>>(dy, ex.down, tiles, pl.max_tiles, s.H, s.I, sv.g, sv.u,
                                                  sv.g_scale, sv.u_scale, dg, du, h);
  else
    k_dh<E, S, false><<<grid, S::THREADS, 0, st>>>(dy, ex.down, tiles, pl.max_tiles, s.H, s.I, sv.g, sv.u,
                                                   nullptr, nullptr, dg, du, h);
  if (const hipError_t e = hipGetLastError()) return e;
  if (drows)
    k_dx<E, S><<<tile_grid(pl, (s.H + S::BN - 1) / S::BN), S::THREADS, 0, st>>>(
        dg, du, ex.gate, ex.up, tiles, pl.max_tiles, s.H, s.I, drows);
  return hipGetLastError();
}

template <class E>
static hipError_t launch_dw(const moe_shape& s, DwArgs& a, hipStream_t st) {
  const auto up = [](int v, int d) { return (v + d - 1) / d; };
  const int it = up(s.I, 128), ht = s.H / 128;
  a.strip = std::min(std::max(3 * s.E * it * ht / 4096, 1), kMaxStrip);
  const int each = 2 * it * up(ht, a.strip) + ht * up(it, a.strip), strips = s.E * each;
  a.unit = std::max(1, std::min(each, strips / 64));
  k_dw<E><<<up(strips, 8 * a.unit) * 8 * a.unit, 256, 0, st>>>(a);
  return hipGetLastError();
}

template <class E>
static hipError_t run_backward(const moe_shape& s, const TrainPlan& pl, const void* dy, const void* x,
                               const uint8_t* x_scale, const moe_saved* sv, const moe_experts& ex,
                               const moe_perm* pm, void* drows, const moe_experts* dex, void* ws,
                               hipStream_t st) {
  const int P = s.T * s.top_k;
  if (P > 0) {
    hipError_t e = launch_prep(s, pl, *pm, ws, st);
    if (e == hipSuccess && dex && x_scale) {
      void* xr = at_off<char>(ws, pl.x_off);
      e = launch_restore8(s.act == MOE_DT_F32, static_cast<size_t>(s.T) * s.H,
                          static_cast<const int8_t*>(x), x_scale, xr, st);
      x = xr;
    }
    if (e == hipSuccess)
      e = pl.bm == Few::BM ? run_rows<E, Few>(s, pl, dy, *sv, ex, drows, ws, st)
                           : run_rows<E, Many>(s, pl, dy, *sv, ex, drows, ws, st);
    if (e != hipSuccess) return e;
  }
  if (!dex) return hipSuccess;
  DwArgs a{};
  a.dy = dy;
  a.x = x;
  a.dgate = const_cast<void*>(dex->gate);
  a.dup = const_cast<void*>(dex->up);
  a.ddown = const_cast<void*>(dex->down);
  a.E = s.E;
  a.H = s.H;
  a.I = s.I;
  a.P = P;
  if (P > 0) {
    a.dg = at_off<char>(ws, pl.dg_off);
    a.du = at_off<char>(ws, pl.du_off);
    a.h = at_off<char>(ws, pl.h_off);
    a.token = at_off<int32_t>(ws, pl.token_off);
    a.offsets = pm->offsets;
  }
  return launch_dw<E>(s, a, st);
}

hipError_t launch_ffn_backward(const moe_shape& s, const TrainPlan& pl, const void* dy,
                               const void* x, const uint8_t* x_scale, const moe_saved* sv,
                               const moe_experts& ex, const moe_perm* pm, void* drows,
                               const moe_experts* dex, void* ws, hipStream_t st) {
  return s.act == MOE_DT_BF16
             ? run_backward<TBf16>(s, pl, dy, x, x_scale, sv, ex, pm, drows, dex, ws, st)
             : run_backward<TF32>(s, pl, dy, x, x_scale, sv, ex, pm, drows, dex, ws, st);
}

}  // namespace moe
