// Prints how the training calls cut their products: for every shape on stdin
//   T H E I k act(0 float32, 1 bf16) t   (t: tiles of 256 rows)
// one line of
//   fits | gate_up: shape parts once tail | dh: shape parts once |
//   dx: shape parts once tail | dw: parts tail | joint
// with shape 0 (32 rows), 1 (128) or 2 (256), tail: into how many parts the last
// 256 x 256 tiles are cut, and dw parts 0 for tiles of 256 x 256.
#include <cstdio>

#include "../sparse_moe_routed_amd/csrc/abi_check.h"
#include "../sparse_moe_routed_amd/csrc/moe_internal.h"

int main() {
  moe_shape s{};
  int t;
  while (std::scanf("%d %d %d %d %d %d %d", &s.T, &s.H, &s.E, &s.I, &s.top_k, &s.act, &t) == 7) {
    moe::TrainPlan p;
    moe::make_train_plan(s, &p);
    const auto up = [](long a, long b) { return static_cast<int>((a + b - 1) / b); };
    const int bk = s.act == MOE_DT_F32 ? 32 : 64;
    const auto tail = [&](bool wide, int slabs, int stages) {
      if (!wide || !moe::Tail::possible(stages)) return 1;
      const auto cut = [&](long tiles) { return moe::Tail(static_cast<int>(tiles * slabs), stages).cut; };
      return s.E == 1 && cut(up(static_cast<long>(s.T) * s.top_k, 256)) < 2 ? 1 : cut(t);
    };
    const long blocks = static_cast<long>(up(s.I, 256)) * up(s.H, 256);
    const int stages = up(static_cast<long>(s.T) * s.top_k / s.E, bk);
    std::printf("%d %d %d %d %d %d %d %d %d %d %d %d %d %d %d\n", moe::train_fits(s, p),
                p.gate_up.shape, p.gate_up.parts, moe::read_once(s, p.gate_up),
                tail(p.gate_up.shape == moe::kRowsWide, up(2 * s.I, 256), s.H / bk),
                p.dh.shape, p.dh.parts, moe::read_once(s, p.dh),
                p.dx.shape, p.dx.parts, moe::read_once(s, p.dx),
                tail(p.dx.shape == moe::kRowsWide, up(s.H, 256), 2 * up(s.I, bk)),
                p.dw_parts, p.dw_parts ? 1 : moe::Tail(static_cast<int>(3 * blocks * s.E), stages).cut, p.joint);
  }
}
