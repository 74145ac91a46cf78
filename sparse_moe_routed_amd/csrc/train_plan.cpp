// Host-side planning of the training calls: tile shapes, splits and the
// workspace layout.  Plain C++ with no device code.
#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "abi_check.h"
#include "moe_internal.h"

namespace moe {

// Tiles of `bm` rows, about: the experts' rows vary around their mean.
static double about_tiles(const moe_shape& s, int bm) {
  const double P = static_cast<double>(s.T) * s.top_k, mean = P / s.E;
  if (mean < 1) return P;
  return s.E * std::max(1.0, static_cast<double>(static_cast<long long>((s.E > 1 ? 1.25 : 1.0) * mean + bm - 1) / bm));
}

// Rounds of 256 x 256 tiles over the CUs, and of those the time of the last ones' joining.
static double wide_us(double tiles, int stages, double each) {
  const Tail t(static_cast<int>(std::min(tiles, 1e9)), stages);
  const double whole = static_cast<double>((t.full + kCus - 1) / kCus);
  return whole * (8 + each * stages) + (t.cut > 1 ? 8 + each * stages / t.cut + 15 : 0);
}

// The cut with the least estimated time.  A product has `columns` columns and a
// sum over `depth`; `half`: a tile has half as many columns (gate beside up).
// Times in us for a stage of 64 bf16 (32 float32) of the sum, measured at 8192
// rows, 2560 x 5120 and 512 experts of 80 rows of 2560 x 640:
//   32 x 128 tiles, four workgroups per CU: 0.6 alone to 1.7 for the four;
//   128 x 256, one per CU: 1.2 (float32 3.6: its matrix rate);
//   256 x 256, one per CU: 1.95 (float32 6.9), only without parts.
// With few tiles the sum is split so that all CUs have work: 64 tokens through
// one block of 2560 x 640 take 40 stages one after the other unsplit.  Joining
// costs a launch and the partial results' way to memory and back.
static RowCut best_cut(const moe_shape& s, int columns, int depth, bool half, bool wide) {
  const bool f32 = s.act == MOE_DT_F32;
  const int stages = (depth * static_cast<int>(act_bytes(s)) + 127) / 128;
  const double P = static_cast<double>(s.T) * s.top_k;
  RowCut best{kRowsFew, 1};
  double least = 1e30;
  for (int shape = kRowsFew; shape <= (wide ? kRowsWide : kRowsMany); ++shape) {
    const int bn = (shape == kRowsFew ? 128 : 256) / (half ? 2 : 1);
    const double groups = about_tiles(s, row_height(shape)) * ((columns + bn - 1) / bn);
    for (int parts : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (parts > 1 && (shape == kRowsWide || stages < 3 * parts)) break;
      const double bytes = 8.0 * parts * P * columns * (half ? 2 : 1);
      if (parts > 1 && bytes > 128e6) break;
      const double n = groups * parts, slots = shape == kRowsFew ? 1024 : 256;
      const double rounds = std::max(1.0, static_cast<double>(static_cast<long long>((n + slots - 1) / slots)));
      const double stage = shape == kRowsFew ? 0.6 + (f32 ? 1.4 : 1.1) * std::min(1.0, n / slots)
                           : shape == kRowsMany ? (f32 ? 3.6 : 1.2) : (f32 ? 6.9 : 1.95);
      const double fixed = shape == kRowsFew ? 2 : 4;
      const double us = shape == kRowsWide ? wide_us(n, stages, stage)
                                           : rounds * (fixed + stage * ((stages + parts - 1) / parts)) +
                                                 (parts > 1 ? 4 + bytes / 5e6 : 0);
      if (us < least) {
        least = us;
        best = RowCut{shape, parts};
      }
    }
  }
  return best;
}

// Parts of an expert's rows in the weight gradients, or 0 for tiles of 256 x 256.
// Times in us for a stage of 64 bf16 (32 float32) rows, measured at 8192 rows, 2560 x
// 5120: 128 x 128 tiles 0.7 alone to 1.5 for the two of a CU (float32 2 to 4), 256 x
// 256, one per CU, 2.05 (float32 7).  One expert's 5000 rows of 2560 x 96 are 60
// tiles of 79 stages: parts give the other CUs work.
static int best_parts(const moe_shape& s) {
  const bool f32 = s.act == MOE_DT_F32;
  const auto up = [](double v, double d) { return static_cast<double>(static_cast<int64_t>((v + d - 1) / d)); };
  const double mean = static_cast<double>(s.T) * s.top_k / s.E, stages = std::max(1.0, up(mean, f32 ? 32 : 64));
  const double values = 3.0 * s.E * s.I * s.H;
  const double tiles = 3 * s.E * up(s.I, 128) * up(s.H, 128), wide = 3 * s.E * up(s.I, 256) * up(s.H, 256);
  int best = 1;
  double least = 1e30;
  for (int parts : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
    const double bytes = 4.0 * parts * values;
    if (parts > 1 && (stages < 2 * parts || bytes > 128e6)) break;
    const double n = tiles * parts, rounds = up(n, 512), both = std::min(1.0, n / 512);
    const double us = rounds * (4 + (f32 ? 2 + 2 * both : 0.7 + 0.8 * both) * up(stages, parts)) +
                      (parts > 1 ? 4 + 2 * bytes / 5e6 : 0);
    if (us < least) {
      least = us;
      best = parts;
    }
  }
  return stages > 2 && wide_us(wide, static_cast<int>(stages), f32 ? 7 : 2.05) < least ? 0 : best;
}

void make_train_plan(const moe_shape& s, TrainPlan* p) {
  const size_t P = static_cast<size_t>(s.T) * s.top_k, a = act_bytes(s);
  *p = TrainPlan{};
  p->dw_parts = best_parts(s);
  if (s.T == 0) return;
  p->gate_up = best_cut(s, s.I, s.H, true, true);
  // its loads and stores after the sum weigh more than what taller tiles save
  // (8192 x 2560 x 5120: 330 us at 128 rows, 384 at 256)
  p->dh = best_cut(s, s.I, s.H, false, false);
  p->dx = best_cut(s, s.H, 2 * s.I, false, true);
  // one list of short tiles serves both products of the gradient
  if (s.E > kLookupExperts && p->dx.shape == kRowsFew && p->dh.shape == kRowsMany) p->dx.shape = kRowsMany;
  if (s.E > kLookupExperts && p->dx.shape == kRowsMany && p->dh.shape == kRowsFew) p->dh.shape = kRowsMany;
  const size_t blocks = (P / row_height(kRowsFew) + std::min<size_t>(s.E, P)) * (s.H / 128);
  p->joint = p->dx.shape == kRowsFew && p->dx.parts == 1 && p->dw_parts == 1 && (blocks + 7) / 8 * 8 <= kJointBlocks;
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t off = at;
    at += align_up(bytes, 256);
    return off;
  };
  for (int list = 0; list < 2; ++list) {
    p->most[list] = static_cast<int>(P / (list ? 256 : 32) + std::min<size_t>(s.E, P));
    p->tiles_off[list] = take(s.E > kLookupExperts ? (static_cast<size_t>(p->most[list]) * 3 + 1) * 4 : 0);
  }
  p->x_off = take(static_cast<size_t>(s.T) * s.H * a);
  p->dg_off = take(P * s.I * a);
  p->du_off = take(P * s.I * a);
  p->h_off = take(P * s.I * a);
  const auto part = [&](const RowCut& c, int columns) {
    return c.parts > 1 ? static_cast<size_t>(c.parts) * P * columns * 4 : 0;
  };
  const auto tail = [](bool wide) { return wide ? static_cast<size_t>(kCus) * kTailBytes : 0; };
  p->rows_part_off = take(std::max({part(p->gate_up, 2 * s.I), part(p->dh, s.I), part(p->dx, s.H),
                                    tail(p->gate_up.shape == kRowsWide || p->dx.shape == kRowsWide)}));
  p->dw_part_off = take(p->dw_parts > 1 ? static_cast<size_t>(p->dw_parts) * 3 * s.E * s.I * s.H * 4 : tail(p->dw_parts == 0));
  const size_t products = at;
  at = 0;
  p->dl_off = take(P * 4);
  p->total = std::max(products, at);
}

bool read_once(const moe_shape& s, const RowCut& c) {
  return static_cast<int64_t>(s.T) * s.top_k <= static_cast<int64_t>(s.E) * row_height(c.shape);
}

bool train_fits(const moe_shape& s, const TrainPlan& p) {
  const uint64_t most = 1u << 23, tiles = static_cast<uint64_t>(p.most[0]);
  if (s.act == MOE_DT_F32 && static_cast<uint64_t>(s.T) * s.H * 4 >= (uint64_t{1} << 32) - 256)
    return false;
  const uint64_t blocks = (s.I + 127) / 128 * static_cast<uint64_t>(s.H / 128);
  return tiles * ((s.I + 63) / 64) < most && tiles * (s.H / 128) < most && 3 * blocks * s.E < most;
}

}  // namespace moe
