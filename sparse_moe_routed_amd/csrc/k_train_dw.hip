// Weight gradients of the routed experts: dW_gate = dg^T x, dW_up = du^T x,
// dW_down = dy^T h, each a sum over the expert's rows.  Both sides of these
// products have their output index contiguous in memory.
#include <algorithm>
#include <type_traits>

#include "train_dw.h"

namespace moe {

// A strip of 128 x 128 tiles of a weight gradient, side by side in n, by four
// waves (64 x 64 each, two workgroups per CU).  M side: dg, du [row][I] or dy
// [row][H]; N side: x of the rows' tokens [token][H], or h [row][I].  Both are
// in columns form, with the expert's rows as k.
//
// An expert of at most two stages of rows keeps its M side in registers for the
// whole strip, and only the N side runs through LDS, step by step of half a
// stage; with more rows both sides run through a ring of two stages.  Either way
// the steps of all tiles are one pipeline, so the next loads are on their way
// while a tile is stored.  PART: float32 sums of a part of the rows.
//
// Bound by the stores: 512 experts of 2560 x 640 are 5.0 GB of gradients, at five
// rows each 920 to 940 us, at 80 skewed ones 1200 (there reads of x, dy and h that
// miss L2, 1.35 GB, compete with them; the fastest of 12 runs, the medians are 985
// and 1250).  Stores of whole cache lines that leave the caches first took 1600 us to
// 1290, steps of half a stage seven deep the five rows from 1100 to 1010.
template <class E, bool PART>
struct DwStrip {
  typedef Shape<2, 2, 4, 2, 16> S;
  typedef std::conditional_t<PART, TF32, E> Out;
  static constexpr int LOADS = 4;                     // of a wave, side and stage
  static constexpr int KR = E::SZ == 2 ? 4 : 2;       // k rows of a load
  static constexpr int PAIR_BYTES = 256;              // of a wave and stage
  static constexpr int LDS = 4 * kBlockBytes + 4 * S::WAVES * PAIR_BYTES;
  static constexpr int STORES = 4 * 16 * Out::SZ / 16;   // of a thread and tile

  const DwArgs& a;
  char* lds;
  Tiles<E, S> T;
  const char *mside, *nside;   // first row of the expert
  char* out;                   // first row of the strip
  bool gather;
  int mcols, ncols, m0, nt0, tiles, row0, rows, stages;
  int krow[LOADS], chunk[LOADS];   // k row and column of this lane's 16 bytes of load j
  u32x4_t pair_rs;
  char* pair_lds;
  int pair_row;
  int lt = 0, ls = 0, ln = 0;   // tile, stage and number of the next loads

  __device__ __forceinline__ DwStrip(const DwArgs& args, char* shared) : a(args), lds(shared) {}

  __device__ __forceinline__ void init(int part, int e, int which, int mt, int first, int count) {
    const bool down = which == 2;
    gather = !down;
    mcols = down ? a.H : a.I;
    ncols = down ? a.I : a.H;
    m0 = mt * 128;
    nt0 = first;
    tiles = count;
    row0 = rows = 0;
    if (a.P > 0) expert_rows(a.offsets, e, a.P, row0, rows);
    if constexpr (PART) {
      const int per = (rows + E::BK * a.parts - 1) / (E::BK * a.parts) * E::BK;
      row0 += min(part * per, rows);
      rows = min(max(rows - part * per, 0), per);
    }
    row0 = __builtin_amdgcn_readfirstlane(row0);
    rows = __builtin_amdgcn_readfirstlane(rows);
    stages = (rows + E::BK - 1) / E::BK;
    mside = static_cast<const char*>(down ? a.dy : which ? a.du : a.dg) +
            (static_cast<size_t>(row0) * mcols + m0) * E::SZ;
    nside = down ? static_cast<const char*>(a.h) + static_cast<size_t>(row0) * a.I * E::SZ
                 : static_cast<const char*>(a.x);
    const size_t whole = static_cast<size_t>(a.I) * a.H, at = static_cast<size_t>(m0) * ncols;
    if constexpr (PART)
      out = reinterpret_cast<char*>(a.part + (static_cast<size_t>(part * 3 + which) * a.E + e) * whole + at);
    else
      out = static_cast<char*>(down ? a.ddown : which ? a.dup : a.dgate) + (e * whole + at) * E::SZ;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      krow[j] = cols_k<E>(j * S::WAVES + T.w, T.lane);
      chunk[j] = (cols_pos<E>(T.lane) ^ key_cols<E>(krow[j])) * (16 / E::SZ);
    }
    // Many rows: the gathered rows' pairs go through LDS too; every wave loads
    // those of its own k rows (lane 8 j + i: row i of load j), with loads n those
    // of loads n + 3.
    pair_rs = buffer(a.sorted_pair + row0);
    pair_lds = lds + 4 * kBlockBytes + T.w * PAIR_BYTES;
    pair_row = cols_k<E>(((T.lane >> 3) & 3) * S::WAVES + T.w, 0) + (T.lane & (KR - 1));
  }

  __device__ __forceinline__ void store_tile(int nt) {
    const char* tile = out + static_cast<size_t>(nt) * 128 * Out::SZ;
#pragma unroll
    for (int t = 0; t < 4; ++t)
      line_pieces<Out>(T.acc[t], T.lane, [&](int row, int col, u32x4_t v) {
        const int r = 64 * T.wm + 16 * t + row, c = 64 * T.wn + col;
        store_piece(tile, nt * 128 + c < ncols && m0 + r < mcols ? static_cast<uint32_t>(r * ncols + c) * Out::SZ : kNowhere, v);
      });
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int f = 0; f < 4; ++f) T.acc[t][f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }

  __device__ __forceinline__ void load_pairs(int s, int slot) const {
    load_lds_word(pair_rs, pair_lds + (slot & 3) * (S::WAVES * PAIR_BYTES),
                  static_cast<uint32_t>(min(s * E::BK + pair_row, rows - 1)) * 4);
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
  // the next N loads, into `st`, and the pairs of those three further on
  __device__ __forceinline__ void issue_n(char* st) {
    const int32_t* tok = reinterpret_cast<const int32_t*>(pair_lds + (ln & 3) * (S::WAVES * PAIR_BYTES));
    const int left = rows - ls * E::BK, n0 = (nt0 + lt) * 128;
    const u32x4_t rn = buffer(nside + (gather ? 0 : static_cast<size_t>(ls) * E::BK * a.I * E::SZ) +
                              static_cast<size_t>(n0) * E::SZ);
    uint32_t off[LOADS];
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const uint32_t token = a.slots.div(min(max(tok[8 * j + (krow[j] & (KR - 1))], 0), a.P - 1));
      const uint32_t row = gather ? token : static_cast<uint32_t>(krow[j]);
      off[j] = krow[j] < left && n0 + chunk[j] < ncols
                   ? row * static_cast<uint32_t>(ncols * E::SZ) + static_cast<uint32_t>(chunk[j] * E::SZ)
                   : kNowhere;
    }
    load_pairs(after(after(after(ls))), ln + 3);
#pragma unroll
    for (int j = 0; j < LOADS; ++j) load_lds(rn, st + (j * S::WAVES + T.w) * 1024, off[j]);
    ++ln;
    if (++ls == stages) {
      ls = 0;
      ++lt;
    }
  }
  __device__ __forceinline__ void first_pairs() const {
    load_pairs(0, 0);
    load_pairs(after(0), 1);
    load_pairs(after(after(0)), 2);
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
      for (int f = 0; f < 4; ++f) T.acc[t][f] = E::mma(n[f], m[t], T.acc[t][f]);
  }

  // At most STEPS (one to four) steps of rows, half a stage each.  The N side's
  // steps of all tiles run through a ring of eight, seven loaded ahead.
  template <int STEPS>
  __device__ __forceinline__ void run_few() {
    constexpr int BYTES = kBlockBytes / 2, RING = 8, AHEAD = RING - 1, PER = LOADS / 2, K = E::BK / 2;
    u32x4_t m[STEPS][4];
    issue_m(0, lds);
    if (STEPS > 2) issue_m(1, lds + kBlockBytes);
    uint32_t off[STEPS][PER];   // byte offset of a lane's 16 bytes within the tile's columns
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int k = s * K + krow[j];
        uint32_t row = k;
        if (gather) row = a.slots.div(min(max(a.sorted_pair[row0 + min(k, rows - 1)], 0), a.P - 1));
        off[s][j] = k < rows ? row * static_cast<uint32_t>(ncols * E::SZ) + static_cast<uint32_t>(chunk[j] * E::SZ) : kNowhere;
      }
    stage_barrier<0>();
#pragma unroll
    for (int s = 0; s < STEPS; ++s) read_m(lds + s * BYTES, 0, m[s]);
    stage_barrier<0>();   // all waves have read
    const int limit = min(ncols, (nt0 + tiles) * 128);   // behind the strip: loads of zeros, to keep count
    const auto issue = [&](int tile, int s, int slot) {
      const int n0 = (nt0 + tile) * 128;
      const u32x4_t rn = buffer(nside + static_cast<size_t>(n0) * E::SZ);
#pragma unroll
      for (int j = 0; j < PER; ++j)
        load_lds(rn, lds + (slot & (RING - 1)) * BYTES + (j * S::WAVES + T.w) * 1024,
                 n0 + chunk[j] < limit ? off[s][j] : kNowhere);
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) issue(i / STEPS, i % STEPS, i);
    int slot = 0;
    for (int t = 0; t < tiles; ++t) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        // This step's loads are done.  Younger are the six after it and the stores of the
        // tiles that ended since they were issued (of all of them or, where a wave's
        // count ends, the last ones).
        constexpr int MOST = (63 - (AHEAD - 1) * PER) / STORES;
        const int stores = std::min((AHEAD - s + STEPS - 1) / STEPS, MOST);
        younger<(AHEAD - 1) * PER>(t < stores ? 0 : stores);
        // all waves have read the step before it
        issue(t + (s + AHEAD) / STEPS, (s + AHEAD) % STEPS, slot + AHEAD);
        u32x4_t n[4];
        read_n(lds + (slot & (RING - 1)) * BYTES, 0, n);
        mma(n, m[s]);
        ++slot;
      }
      store_tile(nt0 + t);
    }
  }
  template <int LOADED>
  static __device__ __forceinline__ void younger(int tiles_stored) {
    switch (tiles_stored) {
      case 0: return stage_barrier<LOADED>();
      case 1: return stage_barrier<LOADED + STORES>();
      case 2: return stage_barrier<LOADED + 2 * STORES>();
      case 3: return stage_barrier<LOADED + 3 * STORES>();
      case 4: return stage_barrier<std::min(63, LOADED + 4 * STORES)>();
      case 5: return stage_barrier<std::min(63, LOADED + 5 * STORES)>();
      default: return stage_barrier<std::min(63, LOADED + 6 * STORES)>();
    }
  }

  // More rows.  The other workgroup of the CU fills the time of this one's reads.
  __device__ __forceinline__ void run_many() {
    const auto issue = [&](char* st) {
      issue_m(ls, st + kBlockBytes);
      issue_n(st);
    };
    first_pairs();
    issue(lds);
    int now = 0;
    for (int t = 0; t < tiles; ++t) {
      for (int s = 0; s < stages; ++s) {
        // younger than this stage's loads: the stores of the tile before
        if (t > 0 && s == 0)
          stage_barrier<STORES>();
        else
          stage_barrier<0>();
        // all waves have read the stage before it
        if (lt < tiles) issue(lds + (now ^ (2 * kBlockBytes)));
        const char* st = lds + now;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          u32x4_t n[4], m[4];
          read_n(st, ks, n);
          read_m(st + kBlockBytes, ks, m);
          mma(n, m);
        }
        now ^= 2 * kBlockBytes;
      }
      store_tile(nt0 + t);
    }
  }
};

template <class E, bool PART>
__device__ __forceinline__ void dw_strip(const DwArgs& a, char* lds, int block) {
  const int it = (a.I + 127) / 128, ht = a.H / 128;
  const int wide = it * ((ht + a.strip - 1) / a.strip), tall = ht * ((it + a.strip - 1) / a.strip);
  const int each = 2 * wide + tall;
  // strips are dealt to the XCDs in units (workgroups in turn)
  const int turn = block >> 3, unit = turn / a.unit;
  int item = (unit * 8 + (block & 7)) * a.unit + turn - unit * a.unit, part = 0;
  if (item >= each * a.E * (PART ? a.parts : 1)) return;
  if constexpr (PART) {
    part = item / (each * a.E);
    item -= part * each * a.E;
  }
  const int e = item / each, in_e = item - e * each;
  const int which = in_e < wide ? 0 : in_e < 2 * wide ? 1 : 2, ntiles = which == 2 ? it : ht;
  const int strips = (ntiles + a.strip - 1) / a.strip, b = in_e - which * wide;
  const int mt = b / strips, nt0 = (b - mt * strips) * a.strip;
  DwStrip<E, PART> s(a, lds);
  s.init(part, e, which, mt, nt0, min(a.strip, ntiles - nt0));
  switch ((s.rows + E::BK / 2 - 1) / (E::BK / 2)) {
    case 0:
      for (int t = 0; t < s.tiles; ++t) s.store_tile(nt0 + t);
      break;
    case 1: s.template run_few<1>(); break;
    case 2: s.template run_few<2>(); break;
    case 3: s.template run_few<3>(); break;
    case 4: s.template run_few<4>(); break;
    default: s.run_many();
  }
}
template <class E, bool PART>
__global__ __launch_bounds__(256, 2) void k_dw(DwArgs a) {
  __shared__ __align__(16) char lds[DwStrip<E, PART>::LDS];
  dw_strip<E, PART>(a, lds, blockIdx.x);
}

// The rows' gradient beside the weights', where it has few tiles: neither needs the
// other, and together they save a launch and the time that the first one's last
// workgroups leave the CUs idle (16 tokens 256 x 64 float32: 21 -> 16 us, 52 tokens
// 2560 x 160 34 -> 25; no difference from 512 workgroups on).
template <class E>
__global__ __launch_bounds__(256, 2) void k_dx_dw(DxArgs x, DwArgs a) {
  __shared__ __align__(16) char lds[DwStrip<E, false>::LDS];
  static_assert(DwStrip<E, false>::LDS >= Few::STAGES * Few::BYTES, "both fit");
  const int block = blockIdx.x;
  if (block < x.blocks)
    dx_tile<E, Few, kOutAct, false>(x.rows, a.dg, a.du, x.gate, x.up, x.drows, lds, block);
  else
    dw_strip<E, false>(a, lds, block - x.blocks);
}

// Joins the parts of all three gradients, eight values a thread.
template <class E>
__global__ __launch_bounds__(256) void k_join_dw(DwArgs a) {
  const size_t each = static_cast<size_t>(a.E) * a.I * a.H;
  const size_t i = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (i >= 3 * each) return;
  float v[8] = {};
  for (int p = 0; p < a.parts; ++p) {
    const float* q = a.part + p * 3 * each + i;
    const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(q), hi = *reinterpret_cast<const f32x4_t*>(q + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] += lo[j];
      v[4 + j] += hi[j];
    }
  }
  const size_t which = i / each;
  store_vals<E>(static_cast<typename E::T*>(which == 2 ? a.ddown : which ? a.dup : a.dgate) + (i - which * each), v);
}

// Many rows per expert: one tile of 256 x 256 by eight waves, both sides through a
// ring of two.
template <class E, bool JOIN>
__global__ __launch_bounds__(512, 2) void k_dw_wide(DwArgs a) {
  typedef Wide S;
  constexpr int KR = E::SZ == 2 ? 4 : 2;          // k rows of a load
  constexpr int PAIRS_LDS = S::WAVES * 256;          // bytes of a stage's tokens, each wave its own
  __shared__ __align__(16) char lds[S::STAGES * S::BYTES + 4 * PAIRS_LDS];
  const int it = (a.I + S::BM - 1) / S::BM, ht = (a.H + S::BM - 1) / S::BM, blocks = it * ht;
  const Tail tail(3 * blocks * a.E, a.mean_stages);
  int item, part = 0, slot, cut = tail.cut;
  if constexpr (JOIN) {
    item = tail.full + blockIdx.x;
    slot = blockIdx.x * cut;
  } else {
    if (!tail.item(blockIdx.x, item, part, slot)) return;
    if (item < tail.full) cut = 1;
  }
  const int e = item / (3 * blocks), in_e = item - e * 3 * blocks, which = in_e / blocks;
  const bool down = which == 2;
  const int mcols = down ? a.H : a.I, ncols = down ? a.I : a.H, ntiles = down ? it : ht;
  const int b = in_e - which * blocks, mt = b / ntiles, nt = b - mt * ntiles;
  int row0 = 0, rows = 0;
  if (a.P > 0) expert_rows(a.offsets, e, a.P, row0, rows);
  row0 = __builtin_amdgcn_readfirstlane(row0);
  rows = __builtin_amdgcn_readfirstlane(rows);

  Tiles<E, S> T;
  const int w = T.w, lane = T.lane, m0 = mt * S::BM, n0 = nt * S::BN;
  const char* mside = static_cast<const char*>(down ? a.dy : which ? a.du : a.dg) +
                      (static_cast<size_t>(row0) * mcols + m0) * E::SZ;
  const char* nside = (down ? static_cast<const char*>(a.h) + static_cast<size_t>(row0) * a.I * E::SZ
                            : static_cast<const char*>(a.x)) + static_cast<size_t>(n0) * E::SZ;
  uint32_t moff[S::ML], noff[S::NL];
  int krow[S::ML];
  T.cols(moff, krow, mcols * E::SZ, mcols - m0);
  T.cols(noff, krow, 0, ncols - n0);   // the rows' own offsets are added stage by stage

  // The gathered rows' pairs go through LDS too, two stages ahead; every wave
  // loads those of its own k rows (lane 8 j + i: row i of loads j and j + 2).
  const u32x4_t rt = buffer(a.sorted_pair + row0);
  char* const pair_lds = lds + S::STAGES * S::BYTES + w * 256;
  const int pair_row = cols_k<E>(((lane >> 3) & 1) * S::WAVES + w, 0) + (lane & (KR - 1));
  const auto load_pairs = [&](int s) {
    load_lds_word(rt, pair_lds + (s & 3) * PAIRS_LDS,
                  static_cast<uint32_t>(max(min(s * E::BK + pair_row, rows - 1), 0)) * 4);
  };
  const int all = (rows + E::BK - 1) / E::BK, s0 = part * all / cut, stages = (part + 1) * all / cut - s0;
  const auto products = [&] { T.run(
      stages, lds,
      [&](int i, char* st) {
        const int s = s0 + i;
        const int left = rows - s * E::BK;
        const int32_t* tok = reinterpret_cast<const int32_t*>(pair_lds + (s & 3) * PAIRS_LDS);
        const u32x4_t rm = buffer(mside + static_cast<size_t>(s) * E::BK * mcols * E::SZ);
        const u32x4_t rn = buffer(nside + (down ? static_cast<size_t>(s) * E::BK * a.I * E::SZ : 0));
        uint32_t off[S::NL];
#pragma unroll
        for (int j = 0; j < S::NL; ++j) {
          const uint32_t token = a.slots.div(min(max(tok[8 * (j & 1) + (krow[j] & (KR - 1))], 0), a.P - 1));
          const uint32_t row = down ? static_cast<uint32_t>(krow[j]) : token;
          off[j] = krow[j] < left && noff[j] != kNowhere ? row * static_cast<uint32_t>(ncols * E::SZ) + noff[j] : kNowhere;
        }
        load_pairs(s + 2);
#pragma unroll
        for (int j = 0; j < S::NL; ++j) T.load_n(j, rn, st, off[j]);
#pragma unroll
        for (int j = 0; j < S::ML; ++j) T.load_m(j, rm, st, krow[j] < left ? moff[j] : kNowhere);
      },
      [&](const char* st, int ks, typename Tiles<E, S>::Frags& f) {
        T.read_n(st, ks, f);
#pragma unroll
        for (int t = 0; t < S::MF; ++t)
          f.m[t] = frag32_cols<E, false>(st + S::NBYTES + T.wm * kBlockBytes, 32 * t, ks, lane);
      }); };
  if constexpr (JOIN) {
    T.add_cuts(a.part, slot, cut);
  } else {
    if (stages > 0) {
      load_pairs(s0);
      load_pairs(s0 + 1);
      stage_barrier<0>();
    }
    products();
    if (cut > 1) return T.store_cut(a.part, slot);
  }

  typename E::T* out = static_cast<typename E::T*>(down ? a.ddown : which ? a.dup : a.dgate) +
                       static_cast<size_t>(e) * a.I * a.H;
#pragma unroll
  for (int t = 0; t < S::MF; ++t) {
    const int r = m0 + T.row(t);
#pragma unroll
    for (int p = 0; p < T.PAIRS; ++p) {
      float v[8];
      T.vals(t, p, v);
      const int c = n0 + T.col(p);
      if (r < mcols && c < ncols) store_vals<E>(out + static_cast<size_t>(r) * ncols + c, v);
    }
  }
}

constexpr int kMaxStrip = 20;

template <class E>
static hipError_t run(const moe_shape& s, DwArgs a, const DxArgs* x, hipStream_t st) {
  const auto up = [](int v, int d) { return (v + d - 1) / d; };
  if (a.parts == 0) {
    const int total = 3 * s.E * up(s.I, Wide::BM) * up(s.H, Wide::BM);
    a.mean_stages = up(a.P / s.E, E::BK);
    const Tail tail(total, a.mean_stages);
    k_dw_wide<E, false><<<up(tail.full, 8) * 8 + up(tail.rest * tail.cut, 8) * 8, Wide::THREADS, 0, st>>>(a);
    if (tail.cut > 1) {
      if (const hipError_t e = hipGetLastError()) return e;
      k_dw_wide<E, true><<<tail.rest, Wide::THREADS, 0, st>>>(a);
    }
    return hipGetLastError();
  }
  const int it = up(s.I, 128), ht = s.H / 128;
  a.strip = std::min(std::max(3 * s.E * it * ht / 4096, 1), kMaxStrip);
  const int each = 2 * it * up(ht, a.strip) + ht * up(it, a.strip), strips = s.E * each * a.parts;
  a.unit = std::max(1, std::min(each, strips / 64));
  const int grid = up(strips, 8 * a.unit) * 8 * a.unit;
  if (a.parts > 1) {
    k_dw<E, true><<<grid, 256, 0, st>>>(a);
    if (const hipError_t e = hipGetLastError()) return e;
    const size_t threads = static_cast<size_t>(3) * s.E * s.I * s.H / 8;
    k_join_dw<E><<<static_cast<int>((threads + 255) / 256), 256, 0, st>>>(a);
  } else if (x) {
    k_dx_dw<E><<<x->blocks + grid, 256, 0, st>>>(*x, a);
  } else {
    k_dw<E, false><<<grid, 256, 0, st>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_dw(const moe_shape& s, const DwArgs& a, const DxArgs* x, hipStream_t st) {
  return s.act == MOE_DT_BF16 ? run<TBf16>(s, a, x, st) : run<TF32>(s, a, x, st);
}

}  // namespace moe
