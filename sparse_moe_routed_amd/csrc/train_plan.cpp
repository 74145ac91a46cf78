// Host-side planning of the training calls: tile heights, splits and the
// workspace layout.  Plain C++ with no device code.
#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "abi_check.h"
#include "moe_internal.h"

namespace moe {

void make_train_plan(const moe_shape& s, TrainPlan* p) {
  const size_t P = static_cast<size_t>(s.T) * s.top_k, a = act_bytes(s);
  *p = TrainPlan{};
  p->bm = P <= static_cast<size_t>(32) * s.E ? 32 : 128;
  p->max_tiles = static_cast<int>(P / p->bm + std::min<size_t>(s.E, P));
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t off = at;
    at += align_up(bytes, 256);
    return off;
  };
  p->tiles_off = take((static_cast<size_t>(p->max_tiles) * 3 + 1) * 4);
  p->token_off = take(P * 4);
  p->x_off = take(static_cast<size_t>(s.T) * s.H * a);
  p->dg_off = take(P * s.I * a);
  p->du_off = take(P * s.I * a);
  p->h_off = take(P * s.I * a);
  const size_t products = at;
  at = 0;
  p->dl_off = take(P * 4);
  p->splits = 1;
  p->part_off = take(p->splits > 1 ? static_cast<size_t>(p->splits) * s.E * (s.H + 1) * 4 : 0);
  p->total = s.T == 0 ? 0 : std::max(products, at);
}

bool train_fits(const moe_shape& s, const TrainPlan& p) {
  const uint64_t most = 1u << 23, tiles = static_cast<uint64_t>(p.max_tiles);
  if (s.act == MOE_DT_F32 && static_cast<uint64_t>(s.T) * s.H * 4 >= (uint64_t{1} << 32) - 256)
    return false;
  const uint64_t blocks = (s.I + 127) / 128 * static_cast<uint64_t>(s.H / 128);
  return tiles * ((s.I + 63) / 64) < most && tiles * (s.H / 128) < most && 3 * blocks * s.E < most;
}

}  // namespace moe
