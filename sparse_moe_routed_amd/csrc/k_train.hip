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

// Offsets of the M side's loads in rows form, MF a wave: `at(row)` gives the
// byte offset of a tile row, rows past the tile are nowhere.
template <int MF, class At>
__device__ __forceinline__ void rows_offsets(uint32_t (&off)[MF], int rows, At&& at) {
  const int w = wave_id(), l = threadIdx.x & 63;
#pragma unroll
  for (int j = 0; j < MF; ++j) {
    const int r = rows_row(j, w, l);
    const uint32_t c = static_cast<uint32_t>(((l & 7) ^ key_rows_m(r)) << 4);
    off[j] = r < rows ? at(r) + c : kNowhere;
  }
}

// ---- gated product ----

// One tile of 32 MF rows x 64 columns of g and of u.  N side: 64 rows of W_gate
// and the same 64 of W_up, so both factors of h end in the same lane.
template <class E, int MF, bool Q8>
__global__ __launch_bounds__(256, 2) void k_gate_up_save(
    const void* __restrict__ x, const void* __restrict__ wg, const void* __restrict__ wu,
    const int32_t* __restrict__ tiles, int max_tiles, const int32_t* __restrict__ token, int H, int I,
    void* __restrict__ g_out, void* __restrict__ u_out, uint8_t* __restrict__ g_scale,
    uint8_t* __restrict__ u_scale, void* __restrict__ h_out) {
  __shared__ __align__(16) char n0[kSideBytes], n1[kSideBytes];
  __shared__ __align__(16) char m0[MF * 4096], m1[MF * 4096];
  TileOf tl;
  if (!tile_of_block(tiles, max_tiles, (I + 63) / 64, tl)) return;
  const int w = wave_id(), lane = threadIdx.x & 63, wn = w & 1, wm = w >> 1;
  const int col0 = tl.slab * 64;
  const size_t wbase = (static_cast<size_t>(tl.e) * I + col0) * H * E::SZ;
  const char* gate = static_cast<const char*>(wg) + wbase;
  const char* up = static_cast<const char*>(wu) + wbase;

  uint32_t moff[MF], noff[2];
  rows_offsets<MF>(moff, tl.rows, [&](int r) {
    return static_cast<uint32_t>(token[tl.row0 + r]) * static_cast<uint32_t>(H * E::SZ);
  });
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = rows_row(j, w, lane);
    noff[j] = col0 + r < I ? static_cast<uint32_t>(r) * (H * E::SZ) +
                                 static_cast<uint32_t>(((lane & 7) ^ key_rows_n(r)) << 4)
                           : kNowhere;
  }

  f32x4_t acc[4][MF] = {};
  stage_loop(
      H / E::BK, n0, m0, n1, m1,
      [&](int s, char* nb, char* mb) {
        const Rsrc rg = buffer(gate + static_cast<size_t>(s) * kStageBytes);
        const Rsrc ru = buffer(up + static_cast<size_t>(s) * kStageBytes);
        const Rsrc rx = buffer(static_cast<const char*>(x) + static_cast<size_t>(s) * kStageBytes);
#pragma unroll
        for (int j = 0; j < 4; ++j) load_lds(j < 2 ? rg : ru, nb + (4 * j + w) * 1024, noff[j & 1]);
#pragma unroll
        for (int j = 0; j < MF; ++j) load_lds(rx, mb + (4 * j + w) * 1024, moff[j]);
      },
      [&](const char* nb, const char* mb) {
#pragma unroll
        for (int ks = 0; ks < E::KS; ++ks) {
          u32x4_t a[4];
#pragma unroll
          for (int f = 0; f < 4; ++f) a[f] = frag_rows_n(nb, wn, f, ks, lane);
#pragma unroll
          for (int t = 0; t < MF; ++t) {
            const u32x4_t b = frag_rows_m(mb, 16 * MF * wm, t, ks, lane);
#pragma unroll
            for (int f = 0; f < 4; ++f) acc[f][t] = E::mma(a[f], b, acc[f][t]);
          }
        }
      });

  // this lane: columns c .. c + 7 of row 16 MF wm + 16 t + i
  const int q = lane >> 4, c = col0 + 32 * wn + 8 * q;
#pragma unroll
  for (int t = 0; t < MF; ++t) {
    const int r = 16 * MF * wm + 16 * t + (lane & 15);
    float g[8], u[8], h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[j] = acc[j >> 2][t][j & 3];
      u[j] = acc[2 + (j >> 2)][t][j & 3];
      h[j] = g[j] / (1.0f + E::exp_neg(g[j])) * u[j];
    }
    uint32_t gs = 0, us = 0;
    if constexpr (Q8) {
      // the largest magnitude as bits: order of magnitude, and NaN above infinity
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

// Offsets of the N side's loads in columns form: k row, column chunk; columns
// past `cols` (from the tile's first column) are nowhere.
template <class E, class Key>
__device__ __forceinline__ uint32_t cols_offset(int j, uint32_t pitch, int cols, Key&& key, int* krow) {
  const int w = wave_id(), l = threadIdx.x & 63;
  const int k = cols_k<E>(j, w, l), chunk = cols_pos<E>(l) ^ key(k);
  *krow = k;
  return chunk * (16 / E::SZ) < cols ? static_cast<uint32_t>(k) * pitch + static_cast<uint32_t>(chunk << 4)
                                     : kNowhere;
}

// dh of one tile of 32 MF rows x 128 columns.
template <class E, int MF, bool Q8>
__global__ __launch_bounds__(256, 2) void k_dh(
    const void* __restrict__ dy, const void* __restrict__ wd, const int32_t* __restrict__ tiles,
    int max_tiles, int H, int I, const void* __restrict__ g_in, const void* __restrict__ u_in,
    const uint8_t* __restrict__ g_scale, const uint8_t* __restrict__ u_scale, void* __restrict__ dg_out,
    void* __restrict__ du_out, void* __restrict__ h_out) {
  __shared__ __align__(16) char n0[kSideBytes], n1[kSideBytes];
  __shared__ __align__(16) char m0[MF * 4096], m1[MF * 4096];
  TileOf tl;
  if (!tile_of_block(tiles, max_tiles, (I + 127) / 128, tl)) return;
  const int w = wave_id(), lane = threadIdx.x & 63, wn = w & 1, wm = w >> 1;
  const int col0 = tl.slab * 128;
  const char* down = static_cast<const char*>(wd) + (static_cast<size_t>(tl.e) * H * I + col0) * E::SZ;
  const char* rows = static_cast<const char*>(dy) + static_cast<size_t>(tl.row0) * H * E::SZ;

  uint32_t moff[MF], noff[4];
  rows_offsets<MF>(moff, tl.rows, [&](int r) { return static_cast<uint32_t>(r) * static_cast<uint32_t>(H * E::SZ); });
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    int k;
    noff[j] = cols_offset<E>(j, I * E::SZ, I - col0, key_cols_n<E>, &k);
  }

  f32x4_t acc[MF][4] = {};
  stage_loop(
      H / E::BK, n0, m0, n1, m1,
      [&](int s, char* nb, char* mb) {
        const Rsrc rn = buffer(down + static_cast<size_t>(s) * E::BK * I * E::SZ);
        const Rsrc rm = buffer(rows + static_cast<size_t>(s) * kStageBytes);
#pragma unroll
        for (int j = 0; j < 4; ++j) load_lds(rn, nb + (4 * j + w) * 1024, noff[j]);
#pragma unroll
        for (int j = 0; j < MF; ++j) load_lds(rm, mb + (4 * j + w) * 1024, moff[j]);
      },
      [&](const char* nb, const char* mb) {
#pragma unroll
        for (int ks = 0; ks < E::KS; ++ks) {
          u32x4_t a[4];
#pragma unroll
          for (int f = 0; f < 4; ++f) a[f] = frag_cols_n<E>(nb, wn, f, ks, lane);
#pragma unroll
          for (int t = 0; t < MF; ++t) {
            const u32x4_t b = frag_rows_m(mb, 16 * MF * wm, t, ks, lane);
#pragma unroll
            for (int f = 0; f < 4; ++f) acc[t][f] = E::mma(a[f], b, acc[t][f]);
          }
        }
      });

  const int c = col0 + 64 * wn + 16 * (lane >> 4);
#pragma unroll
  for (int t = 0; t < MF; ++t) {
    const int r = 16 * MF * wm + 16 * t + (lane & 15);
    if (r >= tl.rows || c >= I) continue;
    const size_t at = static_cast<size_t>(tl.row0 + r) * I + c;
    float dh[16], g[16], u[16], h[16];
    unswap(acc[t], lane, dh);
    if constexpr (Q8) {
      const u32x4_t gc = ld16(static_cast<const char*>(g_in) + at), uc = ld16(static_cast<const char*>(u_in) + at);
      const float gf = factor8(g_scale[at / 32]), uf = factor8(u_scale[at / 32]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        values8(gc[i], gf, g + 4 * i);
        values8(uc[i], uf, u + 4 * i);
      }
    } else {
      load_vals<E>(static_cast<const typename E::T*>(g_in) + at, g);
      load_vals<E>(static_cast<const typename E::T*>(u_in) + at, u);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
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

// ---- gradient: rows ----

// drows of one tile of 32 MF rows x 128 columns: the stages run over I twice,
// dg with W_gate, then du with W_up.
template <class E, int MF>
__global__ __launch_bounds__(256, 2) void k_dx(const void* __restrict__ dg, const void* __restrict__ du,
                                               const void* __restrict__ wg, const void* __restrict__ wu,
                                               const int32_t* __restrict__ tiles, int max_tiles, int H,
                                               int I, void* __restrict__ drows) {
  __shared__ __align__(16) char n0[kSideBytes], n1[kSideBytes];
  __shared__ __align__(16) char m0[MF * 4096], m1[MF * 4096];
  TileOf tl;
  if (!tile_of_block(tiles, max_tiles, H / 128, tl)) return;
  const int w = wave_id(), lane = threadIdx.x & 63, wn = w & 1, wm = w >> 1;
  const int col0 = tl.slab * 128, half = (I + E::BK - 1) / E::BK;
  const size_t wbase = (static_cast<size_t>(tl.e) * I * H + col0) * E::SZ;
  const size_t rbase = static_cast<size_t>(tl.row0) * I * E::SZ;

  uint32_t moff[MF], noff[4];
  rows_offsets<MF>(moff, tl.rows, [&](int r) { return static_cast<uint32_t>(r) * static_cast<uint32_t>(I * E::SZ); });
  const int mchunk = ((lane & 7) ^ key_rows_m(rows_row(0, w, lane))) * (16 / E::SZ);   // the same for every j
  int krow[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) noff[j] = cols_offset<E>(j, H * E::SZ, 128, key_cols_n<E>, &krow[j]);

  f32x4_t acc[MF][4] = {};
  stage_loop(
      2 * half, n0, m0, n1, m1,
      [&](int s, char* nb, char* mb) {
        const int p = s >= half ? s - half : s, left = I - p * E::BK;   // k left from this stage on
        const char* wt = static_cast<const char*>(s >= half ? wu : wg) + wbase;
        const char* dt = static_cast<const char*>(s >= half ? du : dg) + rbase;
        const Rsrc rn = buffer(wt + static_cast<size_t>(p) * E::BK * H * E::SZ);
        const Rsrc rm = buffer(dt + static_cast<size_t>(p) * kStageBytes);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          load_lds(rn, nb + (4 * j + w) * 1024, krow[j] < left ? noff[j] : kNowhere);
#pragma unroll
        for (int j = 0; j < MF; ++j)
          load_lds(rm, mb + (4 * j + w) * 1024, mchunk < left ? moff[j] : kNowhere);
      },
      [&](const char* nb, const char* mb) {
#pragma unroll
        for (int ks = 0; ks < E::KS; ++ks) {
          u32x4_t a[4];
#pragma unroll
          for (int f = 0; f < 4; ++f) a[f] = frag_cols_n<E>(nb, wn, f, ks, lane);
#pragma unroll
          for (int t = 0; t < MF; ++t) {
            const u32x4_t b = frag_rows_m(mb, 16 * MF * wm, t, ks, lane);
#pragma unroll
            for (int f = 0; f < 4; ++f) acc[t][f] = E::mma(a[f], b, acc[t][f]);
          }
        }
      });

  const int c = col0 + 64 * wn + 16 * (lane >> 4);
#pragma unroll
  for (int t = 0; t < MF; ++t) {
    const int r = 16 * MF * wm + 16 * t + (lane & 15);
    if (r >= tl.rows) continue;
    float v[16];
    unswap(acc[t], lane, v);
    store_vals<E>(static_cast<typename E::T*>(drows) + static_cast<size_t>(tl.row0 + r) * H + c, v);
  }
}

// ---- gradient: weights ----

struct DwArgs {
  const void *dg, *du, *h, *dy, *x;
  void *dgate, *dup, *ddown;
  const int32_t *offsets, *token;
  int E, H, I, P;
};

// One 128 x 128 tile of a weight gradient.  M side: dg, du [row][I] or dy
// [row][H]; N side: x of the rows' tokens [token][H], or h [row][I].
template <class E>
__global__ __launch_bounds__(256, 2) void k_dw(DwArgs a) {
  __shared__ __align__(16) char n0[kSideBytes], n1[kSideBytes];
  __shared__ __align__(16) char m0[kSideBytes], m1[kSideBytes];
  const int it = (a.I + 127) / 128, ht = a.H / 128, blocks = it * ht;
  const int total = 3 * blocks * a.E, per = (total + 7) / 8, s8 = static_cast<int>(blockIdx.x >> 3);
  const int item = static_cast<int>(blockIdx.x & 7) * per + s8;
  if (s8 >= per || item >= total) return;
  const int e = item / (3 * blocks), in_e = item - e * 3 * blocks, which = in_e / blocks;
  const int b = in_e - which * blocks;
  const bool is_down = which == 2;
  const int mcols = is_down ? a.H : a.I, ncols = is_down ? a.I : a.H;
  const int ntiles = is_down ? it : ht;
  const int mt = b / ntiles, nt = b - mt * ntiles;
  int row0 = 0, rows = 0;
  if (a.P > 0) expert_rows(a.offsets, e, a.P, row0, rows);
  row0 = __builtin_amdgcn_readfirstlane(row0);
  rows = __builtin_amdgcn_readfirstlane(rows);

  const int w = wave_id(), lane = threadIdx.x & 63, wn = w & 1, wm = w >> 1;
  const char* mside = static_cast<const char*>(is_down ? a.dy : which ? a.du : a.dg) +
                      (static_cast<size_t>(row0) * mcols + mt * 128) * E::SZ;
  const char* nside = is_down ? static_cast<const char*>(a.h) + (static_cast<size_t>(row0) * a.I + nt * 128) * E::SZ
                              : static_cast<const char*>(a.x) + static_cast<size_t>(nt) * 128 * E::SZ;
  uint32_t moff[4], noff[4], tok[4];
  int krow[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    moff[j] = cols_offset<E>(j, mcols * E::SZ, mcols - mt * 128, key_cols_m<E>, &krow[j]);
    // the gathered rows' offset is added stage by stage
    noff[j] = cols_offset<E>(j, is_down ? ncols * E::SZ : 0, ncols - nt * 128, key_cols_n<E>, &krow[j]);
  }
  const auto tokens = [&](int s) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = s * E::BK + krow[j];
      tok[j] = !is_down && r < rows ? static_cast<uint32_t>(a.token[row0 + r]) : 0u;
    }
  };
  tokens(0);

  f32x4_t acc[4][4] = {};
  stage_loop(
      (rows + E::BK - 1) / E::BK, n0, m0, n1, m1,
      [&](int s, char* nb, char* mb) {
        const int left = rows - s * E::BK;
        const Rsrc rm = buffer(mside + static_cast<size_t>(s) * E::BK * mcols * E::SZ);
        const Rsrc rn = buffer(is_down ? nside + static_cast<size_t>(s) * E::BK * a.I * E::SZ : nside);
#pragma unroll
        for (int j = 0; j < 4; ++j) load_lds(rm, mb + (4 * j + w) * 1024, krow[j] < left ? moff[j] : kNowhere);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool on = krow[j] < left && noff[j] != kNowhere;
          load_lds(rn, nb + (4 * j + w) * 1024,
                   on ? noff[j] + tok[j] * static_cast<uint32_t>(a.H * E::SZ) : kNowhere);
        }
        tokens(s + 1);
      },
      [&](const char* nb, const char* mb) {
#pragma unroll
        for (int ks = 0; ks < E::KS; ++ks) {
          u32x4_t f4[4];
#pragma unroll
          for (int f = 0; f < 4; ++f) f4[f] = frag_cols_n<E>(nb, wn, f, ks, lane);
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const u32x4_t b4 = frag_cols_m<E>(mb, wm, t, ks, lane);
#pragma unroll
            for (int f = 0; f < 4; ++f) acc[t][f] = E::mma(f4[f], b4, acc[t][f]);
          }
        }
      });

  typename E::T* out = static_cast<typename E::T*>(is_down ? a.ddown : which ? a.dup : a.dgate) +
                       static_cast<size_t>(e) * a.I * a.H;
  const int c = nt * 128 + 64 * wn + 16 * (lane >> 4);
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int r = mt * 128 + 64 * wm + 16 * t + (lane & 15);
    if (r >= mcols || c >= ncols) continue;
    float v[16];
    unswap(acc[t], lane, v);
    store_vals<E>(out + static_cast<size_t>(r) * ncols + c, v);
  }
}

// ---- launches ----

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

template <class E, int MF, bool Q8>
static void run_gate_up(const moe_shape& s, const TrainPlan& pl, const void* x, const moe_experts& ex,
                        const moe_saved& sv, void* h, void* ws, hipStream_t st) {
  k_gate_up_save<E, MF, Q8><<<tile_grid(pl, (s.I + 63) / 64), 256, 0, st>>>(
      x, ex.gate, ex.up, at_off<int32_t>(ws, pl.tiles_off), pl.max_tiles, at_off<int32_t>(ws, pl.token_off),
      s.H, s.I, sv.g, sv.u, sv.g_scale, sv.u_scale, h);
}

template <class E>
static void run_gate_up(const moe_shape& s, const TrainPlan& pl, const void* x, const moe_experts& ex,
                        const moe_saved& sv, void* h, void* ws, hipStream_t st) {
  const bool q8 = sv.g_scale != nullptr;
  if (pl.bm == 32)
    q8 ? run_gate_up<E, 1, true>(s, pl, x, ex, sv, h, ws, st) : run_gate_up<E, 1, false>(s, pl, x, ex, sv, h, ws, st);
  else
    q8 ? run_gate_up<E, 4, true>(s, pl, x, ex, sv, h, ws, st) : run_gate_up<E, 4, false>(s, pl, x, ex, sv, h, ws, st);
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

template <class E, int MF>
static hipError_t run_rows(const moe_shape& s, const TrainPlan& pl, const void* dy, const moe_saved& sv,
                           const moe_experts& ex, void* drows, void* ws, hipStream_t st) {
  const int32_t* tiles = at_off<int32_t>(ws, pl.tiles_off);
  void *dg = at_off<char>(ws, pl.dg_off), *du = at_off<char>(ws, pl.du_off), *h = at_off<char>(ws, pl.h_off);
  const int grid = tile_grid(pl, (s.I + 127) / 128);
  if (sv.g_scale)
    k_dh<E, MF, true><<<grid, 256, 0, st>>>(dy, ex.down, tiles, pl.max_tiles, s.H, s.I, sv.g, sv.u,
                                            sv.g_scale, sv.u_scale, dg, du, h);
  else
    k_dh<E, MF, false><<<grid, 256, 0, st>>>(dy, ex.down, tiles, pl.max_tiles, s.H, s.I, sv.g, sv.u,
                                             nullptr, nullptr, dg, du, h);
  if (const hipError_t e = hipGetLastError()) return e;
  if (drows)
    k_dx<E, MF><<<tile_grid(pl, s.H / 128), 256, 0, st>>>(dg, du, ex.gate, ex.up, tiles, pl.max_tiles, s.H,
                                                          s.I, drows);
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
      e = pl.bm == 32 ? run_rows<E, 1>(s, pl, dy, *sv, ex, drows, ws, st)
                      : run_rows<E, 4>(s, pl, dy, *sv, ex, drows, ws, st);
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
  const int total = 3 * s.E * ((s.I + 127) / 128) * (s.H / 128);
  k_dw<E><<<(total + 7) / 8 * 8, 256, 0, st>>>(a);
  return hipGetLastError();
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
