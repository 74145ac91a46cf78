// Training of the routed experts: preparation and launches of the gated product
// that keeps g and u, and of the gradient of the gated product and the down
// projection (kernels: train_rows.h, k_train_dw.hip).
#include "moe_internal.h"
#include "train_dw.h"
#include "train_rows.h"

namespace moe {

// Tile list of one row height, for more experts than a wave has lanes.  Every
// thread finds the experts of its tiles in the running numbers of tiles.
struct TileList {
  int32_t* tiles;
  int most, bm;
};
__global__ __launch_bounds__(1024) void k_train_tiles(const int32_t* __restrict__ offsets, int E, int P,
                                                      TileList first, TileList second) {
  const TileList l = blockIdx.x ? second : first;
  __shared__ int sums[16];
  __shared__ int before[1024];   // tiles of the experts before this one
  const int e = threadIdx.x, lane = e & 63, w = e >> 6;
  int row0 = 0, rows = 0;
  if (e < E) expert_rows(offsets, e, P, row0, rows);
  const int n = (rows + l.bm - 1) / l.bm, incl = wave_incl_scan_i32(n);
  if (lane == 63) sums[w] = incl;
  __syncthreads();
  int at = incl - n, all = 0;
  for (int i = 0; i < 16; ++i) {
    if (i < w) at += sums[i];
    all += sums[i];
  }
  before[e] = at;
  __syncthreads();
  all = min(all, l.most);
  if (e == 0) l.tiles[3 * l.most] = all;
  for (int t = threadIdx.x; t < all; t += 1024) {
    int lo = 0, hi = E;   // before[lo] <= t < before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      (before[mid] <= t ? lo : hi) = mid;
    }
    int r0, r;
    expert_rows(offsets, lo, P, r0, r);
    const int j = t - before[lo];
    l.tiles[3 * t] = lo;
    l.tiles[3 * t + 1] = r0 + j * l.bm;
    l.tiles[3 * t + 2] = min(r - j * l.bm, l.bm);
  }
}

static int list_of(const RowCut& c) { return c.shape == kRowsWide ? 1 : 0; }

static RowArgs row_args(const moe_shape& s, const TrainPlan& pl, const moe_perm& pm, void* ws, const RowCut& c) {
  RowArgs a{};
  const int l = list_of(c);
  if (s.E > kLookupExperts) a.tiles = at_off<int32_t>(ws, pl.tiles_off[l]);
  a.most = pl.most[l];
  a.offsets = pm.offsets;
  a.sorted_pair = pm.sorted_pair;
  a.part = at_off<float>(ws, pl.rows_part_off);
  a.E = s.E;
  a.H = s.H;
  a.I = s.I;
  a.P = s.T * s.top_k;
  a.parts = c.parts;
  a.slots = PairDiv::of(s.top_k);
  return a;
}

// Writes the tile lists of the heights that a call's cuts need: at most one of
// 32 and 128, and 256.
static hipError_t launch_tiles(const moe_shape& s, const TrainPlan& pl, const moe_perm& pm, void* ws, int small,
                               bool wide, hipStream_t st) {
  if (s.E <= kLookupExperts) return hipSuccess;
  const TileList first{at_off<int32_t>(ws, pl.tiles_off[0]), pl.most[0], small};
  const TileList second{at_off<int32_t>(ws, pl.tiles_off[1]), pl.most[1], 256};
  k_train_tiles<<<small && wide ? 2 : 1, 1024, 0, st>>>(pm.offsets, s.E, s.T * s.top_k, small ? first : second, second);
  return hipGetLastError();
}

// f(shape) of a cut.
template <bool WIDE, class F>
static hipError_t with_shape(const moe_shape& s, const RowCut& c, F&& f) {
  const bool once = read_once(s, c);
  if (c.shape == kRowsWide) {
    if constexpr (WIDE) return f(Wide{});
    return hipErrorInvalidValue;   // a product that is not made in this shape
  }
  if (c.shape == kRowsFew) return once ? f(FewOnce{}) : f(Few{});
  return once ? f(ManyOnce{}) : f(Many{});
}

template <class E>
static hipError_t gate_up(const moe_shape& s, const TrainPlan& pl, const void* x, const moe_experts& ex,
                          const moe_perm& pm, const moe_saved& sv, void* h, void* ws, hipStream_t st) {
  const RowArgs a = row_args(s, pl, pm, ws, pl.gate_up);
  const GateUpOut o{sv.g, sv.u, h, sv.g_scale, sv.u_scale};
  return with_shape<true>(s, pl.gate_up, [&](auto shape) { return run_gate_up<E, decltype(shape)>(a, x, ex, o, st); });
}

hipError_t launch_gate_up_save(const moe_shape& s, const TrainPlan& pl, const void* x,
                               const moe_experts& ex, const moe_perm& pm, const moe_saved& sv,
                               void* h, void* ws, hipStream_t st) {
  const int l = list_of(pl.gate_up);
  if (const hipError_t e = launch_tiles(s, pl, pm, ws, l ? 0 : row_height(pl.gate_up.shape), l, st)) return e;
  return s.act == MOE_DT_BF16 ? gate_up<TBf16>(s, pl, x, ex, pm, sv, h, ws, st)
                              : gate_up<TF32>(s, pl, x, ex, pm, sv, h, ws, st);
}

template <class E>
static hipError_t rows_backward(const moe_shape& s, const TrainPlan& pl, const void* dy, const DhArgs& d,
                                const moe_experts& ex, const moe_perm& pm, void* drows, void* ws, hipStream_t st) {
  const RowArgs a = row_args(s, pl, pm, ws, pl.dh), b = row_args(s, pl, pm, ws, pl.dx);
  const hipError_t e =
      with_shape<false>(s, pl.dh, [&](auto shape) { return run_dh<E, decltype(shape)>(a, dy, ex.down, d, st); });
  if (e != hipSuccess || !drows) return e;
  return with_shape<true>(s, pl.dx, [&](auto shape) { return run_dx<E, decltype(shape)>(b, d, ex, drows, st); });
}

hipError_t launch_ffn_backward(const moe_shape& s, const TrainPlan& pl, const void* dy,
                               const void* x, const uint8_t* x_scale, const moe_saved* sv,
                               const moe_experts& ex, const moe_perm* pm, void* drows,
                               const moe_experts* dex, void* ws, hipStream_t st) {
  const bool bf16 = s.act == MOE_DT_BF16;
  DwArgs a{};
  DxArgs dx{};
  bool joint = false;
  a.E = s.E;
  a.H = s.H;
  a.I = s.I;
  a.P = s.T * s.top_k;
  if (a.P > 0) {
    const bool wide = drows && pl.dx.shape == kRowsWide;
    hipError_t e = launch_tiles(s, pl, *pm, ws, row_height(pl.dh.shape), wide, st);
    if (e == hipSuccess && dex && x_scale) {
      void* xr = at_off<char>(ws, pl.x_off);
      e = launch_restore8(!bf16, static_cast<size_t>(s.T) * s.H, static_cast<const int8_t*>(x), x_scale, xr, st);
      x = xr;
    }
    const DhArgs d{sv->g, sv->u, sv->g_scale, sv->u_scale, at_off<char>(ws, pl.dg_off), at_off<char>(ws, pl.du_off),
                   at_off<char>(ws, pl.h_off)};
    joint = drows && dex && pl.joint;
    if (joint) {
      dx.rows = row_args(s, pl, *pm, ws, pl.dx);
      dx.gate = ex.gate;
      dx.up = ex.up;
      dx.drows = drows;
      dx.blocks = tile_grid<Few>(dx.rows, s.H / 128);
      drows = nullptr;
    }
    if (e == hipSuccess)
      e = bf16 ? rows_backward<TBf16>(s, pl, dy, d, ex, *pm, drows, ws, st)
               : rows_backward<TF32>(s, pl, dy, d, ex, *pm, drows, ws, st);
    if (e != hipSuccess) return e;
    a.dg = d.dg;
    a.du = d.du;
    a.h = d.h;
    a.offsets = pm->offsets;
    a.sorted_pair = pm->sorted_pair;
    a.slots = PairDiv::of(s.top_k);
  }
  if (!dex) return hipSuccess;
  a.parts = pl.dw_parts;
  a.part = at_off<float>(ws, pl.dw_part_off);
  a.dy = dy;
  a.x = x;
  a.dgate = const_cast<void*>(dex->gate);
  a.dup = const_cast<void*>(dex->up);
  a.ddown = const_cast<void*>(dex->down);
  return launch_dw(s, a, joint ? &dx : nullptr, st);
}

}  // namespace moe
