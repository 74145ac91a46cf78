// Weight gradients of the routed experts: dW_gate = dg^T x, dW_up = du^T x,
// dW_down = dy^T h, each a sum over the expert's rows.  Both sides of these
// products have their output index contiguous in memory.
#include <algorithm>

#include "train_dw.h"

namespace moe {

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
  typedef Shape<2, 2, 4, 2, 16> S;
  static constexpr int LOADS = 4;                     // of a wave, side and stage
  static constexpr int KR = E::SZ == 2 ? 4 : 2;       // k rows of a load
  static constexpr int PAIR_BYTES = 256;             // of a wave and stage
  static constexpr int LDS = 4 * kBlockBytes + 4 * S::WAVES * PAIR_BYTES;
  static constexpr int STORES = 4 * 16 * E::SZ / 16;  // of a thread and tile

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
    // The gathered rows' pairs go through LDS too; every wave loads those of its
    // own k rows (lane 8 j + i: row i of load j).  Those of loads n are requested
    // with loads n - 3: loads n are issued when loads n - 3 (few rows) or later
    // ones (many rows) are known to have landed.
    pair_rs = buffer(a.sorted_pair + row0);
    pair_lds = lds + 4 * kBlockBytes + T.w * PAIR_BYTES;
    pair_row = cols_k<E>(((T.lane >> 3) & 3) * S::WAVES + T.w, 0) + (T.lane & (KR - 1));
  }

  __device__ __forceinline__ void store_tile(int nt) {
    const char* tile = out + static_cast<size_t>(nt) * 128 * E::SZ;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int r = T.row(t);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        float v[8];
        pair_vals(T.acc[t], p, v);
        const int c = T.col(p);
        store_vals<E>(tile, nt * 128 + c < ncols && m0 + r < mcols ? static_cast<uint32_t>(r * ncols + c) * E::SZ : kNowhere, v);
      }
    }
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

  // at most two stages of rows
  __device__ __forceinline__ void run_few() {
    u32x4_t m[2][2][4];   // stage, step
    first_pairs();
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
    first_pairs();
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

// Many rows per expert: one tile of 256 x 256 by eight waves, both sides through a
// ring of two.
template <class E>
__global__ __launch_bounds__(512, 2) void k_dw_wide(DwArgs a) {
  typedef Wide S;
  constexpr int KR = E::SZ == 2 ? 4 : 2;          // k rows of a load
  constexpr int PAIRS_LDS = S::WAVES * 256;          // bytes of a stage's tokens, each wave its own
  __shared__ __align__(16) char lds[S::STAGES * S::BYTES + 4 * PAIRS_LDS];
  const int it = (a.I + S::BM - 1) / S::BM, ht = (a.H + S::BM - 1) / S::BM, blocks = it * ht;
  const int total = 3 * blocks * a.E, per = (total + 7) / 8, turn = static_cast<int>(blockIdx.x >> 3);
  const int item = static_cast<int>(blockIdx.x & 7) * per + turn;
  if (turn >= per || item >= total) return;
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
  const int stages = (rows + E::BK - 1) / E::BK;
  if (stages > 0) {
    load_pairs(0);
    load_pairs(1);
    stage_barrier<0>();
  }
  T.run(
      stages, lds,
      [&](int s, char* st) {
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
      });

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
static hipError_t run(const moe_shape& s, DwArgs a, hipStream_t st) {
  const auto up = [](int v, int d) { return (v + d - 1) / d; };
  if (a.P / s.E >= 512) {
    const int total = 3 * s.E * up(s.I, Wide::BM) * up(s.H, Wide::BM);
    k_dw_wide<E><<<up(total, 8) * 8, Wide::THREADS, 0, st>>>(a);
    return hipGetLastError();
  }
  const int it = up(s.I, 128), ht = s.H / 128;
  a.strip = std::min(std::max(3 * s.E * it * ht / 4096, 1), kMaxStrip);
  const int each = 2 * it * up(ht, a.strip) + ht * up(it, a.strip), strips = s.E * each;
  a.unit = std::max(1, std::min(each, strips / 64));
  k_dw<E><<<up(strips, 8 * a.unit) * 8 * a.unit, 256, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_dw(const moe_shape& s, const DwArgs& a, hipStream_t st) {
  return s.act == MOE_DT_BF16 ? run<TBf16>(s, a, st) : run<TF32>(s, a, st);
}

}  // namespace moe
