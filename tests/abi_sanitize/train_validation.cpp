// Host-only validation battery of the training calls (train_abi.cpp), built
// with AddressSanitizer and UndefinedBehaviorSanitizer and launchers that abort
// if reached: every call below must be refused (or is an empty batch), reach
// no launcher and leave its sentinel buffers alone.  Workspace sizes are
// computed over the corners of the domain.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <limits>
#include <vector>

#include "../../sparse_moe_routed_amd/csrc/moe_internal.h"

namespace moe {

[[noreturn]] static void reached(const char* name) {
  std::fprintf(stderr, "FAIL: %s was reached by a call that must be rejected\n", name);
  std::abort();
}

hipError_t launch_save8(bool, size_t, const void*, int8_t*, uint8_t*, hipStream_t) { reached("launch_save8"); }
hipError_t launch_restore8(bool, size_t, const int8_t*, const uint8_t*, void*, hipStream_t) {
  reached("launch_restore8");
}
hipError_t launch_gate_up_save(const moe_shape&, const TrainPlan&, const void*, const moe_experts&,
                               const moe_perm&, const moe_saved&, void*, void*, hipStream_t) {
  reached("launch_gate_up_save");
}
hipError_t launch_ffn_backward(const moe_shape&, const TrainPlan&, const void*, const void*,
                               const uint8_t*, const moe_saved*, const moe_experts&, const moe_perm*,
                               void*, const moe_experts*, void*, hipStream_t) {
  reached("launch_ffn_backward");
}
hipError_t launch_router_bwd(const moe_shape&, const RouterBwd&, hipStream_t) {
  reached("launch_router_bwd");
}

}  // namespace moe

namespace {

int g_fail = 0;

void expect(int line, long got, long want) {
  if (got == want) return;
  std::fprintf(stderr, "FAIL %s:%d: %ld, want %ld\n", __FILE__, line, got, want);
  ++g_fail;
}
#define EXPECT(call, want) expect(__LINE__, (call), (want))

struct Buf {
  std::vector<unsigned char> a;
  unsigned char* p;
  explicit Buf(size_t n) : a(n + 512, 0xA5) {
    p = a.data() + (256 - reinterpret_cast<uintptr_t>(a.data()) % 256) % 256;
  }
  bool untouched() const {
    for (unsigned char c : a)
      if (c != 0xA5) return false;
    return true;
  }
};

struct Set {
  std::vector<Buf> b;
  Set() {
    b.reserve(20);
    for (int i = 0; i < 20; ++i) b.emplace_back(1 << 17);
  }
  void* operator[](int i) { return b[i].p; }
  bool untouched() const {
    for (const Buf& x : b)
      if (!x.untouched()) return false;
    return true;
  }
};

moe_shape shape(int T, int H, int E, int I, int k, int act = MOE_DT_BF16, int wfmt = MOE_WF_DENSE,
                uint32_t flags = 0) {
  return moe_shape{T, H, E, I, k, act, wfmt, flags};
}

void sizes() {
  const int big = std::numeric_limits<int>::max();
  for (int T : {-1, 0, 1, 131072, 131073, big})
    for (int H : {0, 128, 100, 65536, 65664, big})
      for (int E : {0, 1, 1024, 1025, big})
        for (int I : {0, 32, 33, 65536, big})
          for (int k : {0, 1, 10, 1024, big})
            for (int act : {0, 1, 7}) {
              const moe_shape s = shape(T, H, E, I, k, act);
              const size_t n = moe_train_workspace_size(&s);
              if (moe::check_shape(&s) != MOE_OK || T == 0) {
                EXPECT(n != 0, 0);
                continue;
              }
              const size_t P = static_cast<size_t>(T) * k, a = act == MOE_DT_F32 ? 4 : 2;
              EXPECT(n >= 3 * P * I * a + static_cast<size_t>(T) * H * a, 1);
              moe::TrainPlan pl;
              moe::make_train_plan(s, &pl);
              for (const moe::RowCut& c : {pl.gate_up, pl.dh, pl.dx}) EXPECT(c.shape >= 0 && c.shape <= 2 && c.parts >= 1, 1);
              EXPECT(pl.most[0] >= 1 && pl.most[1] >= 1, 1);
              (void)moe::train_fits(s, pl);
            }
}

void refusals() {
  Set b;
  moe_shape s = shape(4, 128, 8, 64, 2);
  const size_t ws = moe_train_workspace_size(&s);
  const auto i32 = [&](int i) { return static_cast<int32_t*>(b[i]); };
  const auto f32 = [&](int i) { return static_cast<float*>(b[i]); };
  const auto u8 = [&](int i) { return static_cast<uint8_t*>(b[i]); };
  const moe_experts ex{b[0], b[1], b[2], nullptr, nullptr, nullptr};
  const moe_experts dex{b[3], b[4], b[5], nullptr, nullptr, nullptr};
  const moe_perm pm{nullptr, i32(6), i32(7), nullptr, nullptr, nullptr};
  const moe_saved sv{b[8], b[9], u8(10), u8(11)};

  // nothing where something is needed, a workspace too small, outputs on inputs
  EXPECT(moe_ffn_gate_up_save(&s, b[12], &ex, &pm, &sv, b[13], b[14], ws - 1, nullptr), MOE_E_WORKSPACE);
  EXPECT(moe_ffn_gate_up_save(&s, b[12], &ex, &pm, &sv, b[12], b[14], ws, nullptr), MOE_E_ALIAS);
  EXPECT(moe_ffn_gate_up_save(&s, b[12], &ex, &pm, &sv, b[8], b[14], ws, nullptr), MOE_E_ALIAS);
  EXPECT(moe_ffn_gate_up_save(&s, b[12], &ex, &pm, &sv, b[13], b[0], ws, nullptr), MOE_E_ALIAS);
  EXPECT(moe_ffn_gate_up_save(&s, nullptr, &ex, &pm, &sv, b[13], b[14], ws, nullptr), MOE_E_NULL);
  EXPECT(moe_ffn_gate_up_save(nullptr, b[12], &ex, &pm, &sv, b[13], b[14], ws, nullptr), MOE_E_NULL);
  EXPECT(moe_ffn_gate_up_save(&s, b[12], nullptr, &pm, &sv, b[13], b[14], ws, nullptr), MOE_E_NULL);
  EXPECT(moe_ffn_gate_up_save(&s, b[12], &ex, nullptr, &sv, b[13], b[14], ws, nullptr), MOE_E_NULL);
  EXPECT(moe_ffn_gate_up_save(&s, b[12], &ex, &pm, nullptr, b[13], b[14], ws, nullptr), MOE_E_NULL);

  EXPECT(moe_ffn_backward(&s, b[12], b[13], u8(14), &sv, &ex, &pm, b[15], &dex, b[16], ws - 1, nullptr), MOE_E_WORKSPACE);
  EXPECT(moe_ffn_backward(&s, b[12], b[13], u8(14), &sv, &ex, &pm, b[12], &dex, b[16], ws, nullptr), MOE_E_ALIAS);
  EXPECT(moe_ffn_backward(&s, b[12], b[13], u8(14), &sv, &ex, &pm, b[15], &ex, b[16], ws, nullptr), MOE_E_ALIAS);
  EXPECT(moe_ffn_backward(&s, b[12], b[13], u8(14), &sv, &ex, &pm, b[15], &dex, b[14], ws, nullptr), MOE_E_ALIAS);
  EXPECT(moe_ffn_backward(&s, b[12], b[13], u8(14), &sv, &ex, &pm, nullptr, nullptr, b[16], ws, nullptr), MOE_E_NULL);
  EXPECT(moe_ffn_backward(&s, b[12], nullptr, nullptr, &sv, &ex, &pm, b[15], &dex, b[16], ws, nullptr), MOE_E_NULL);
  EXPECT(moe_ffn_backward(&s, nullptr, b[13], nullptr, &sv, &ex, &pm, b[15], &dex, b[16], ws, nullptr), MOE_E_NULL);
  EXPECT(moe_ffn_backward(&s, b[12], b[13], nullptr, nullptr, &ex, &pm, b[15], &dex, b[16], ws, nullptr), MOE_E_NULL);
  EXPECT(moe_ffn_backward(&s, b[12], b[13], nullptr, &sv, nullptr, &pm, b[15], &dex, b[16], ws, nullptr), MOE_E_NULL);
  EXPECT(moe_ffn_backward(&s, b[12], b[13], nullptr, &sv, &ex, nullptr, b[15], &dex, b[16], ws, nullptr), MOE_E_NULL);
  moe_shape t = s;
  t.T = 0;
  EXPECT(moe_ffn_backward(&t, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, b[15], nullptr, nullptr, 0, nullptr), MOE_OK);
  EXPECT(moe_ffn_gate_up_save(&t, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr), MOE_OK);

  EXPECT(moe_router_backward(&s, i32(12), f32(13), f32(14), b[15], b[0], &pm, nullptr, b[16], f32(17), f32(18),
                             b[19], ws - 1, nullptr), MOE_E_WORKSPACE);
  EXPECT(moe_router_backward(&s, i32(12), f32(13), f32(14), b[15], b[0], &pm, b[1], b[1], f32(17), f32(18),
                             b[19], ws, nullptr), MOE_E_ALIAS);
  EXPECT(moe_router_backward(&s, i32(12), f32(13), f32(14), b[15], b[0], nullptr, nullptr, b[16], f32(17), nullptr,
                             b[19], ws, nullptr), MOE_E_NULL);
  EXPECT(moe_router_backward(&t, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, b[16], nullptr,
                             nullptr, nullptr, 0, nullptr), MOE_OK);

  for (int64_t rows : {int64_t{-1}, int64_t{0}, int64_t{8}, int64_t{1} << 40, std::numeric_limits<int64_t>::max()})
    for (int64_t cols : {int64_t{-32}, int64_t{0}, int64_t{31}, int64_t{32}, std::numeric_limits<int64_t>::max() / 32 * 32}) {
      const int want = rows < 0 || cols < 32 || cols % 32 ? MOE_E_SHAPE
                       : rows > (int64_t{1} << 40) / cols ? MOE_E_LIMIT
                       : rows == 0                        ? MOE_OK
                                                          : MOE_E_NULL;
      EXPECT(moe_save8(MOE_DT_BF16, rows, cols, nullptr, nullptr, nullptr, nullptr), want);
      EXPECT(moe_restore8(MOE_DT_F32, rows, cols, nullptr, nullptr, nullptr, nullptr), want);
    }
  EXPECT(moe_save8(9, 8, 64, b[0], static_cast<int8_t*>(b[1]), u8(2), nullptr), MOE_E_DTYPE);
  EXPECT(moe_save8(MOE_DT_BF16, 8, 64, b[0], static_cast<int8_t*>(b[0]), u8(2), nullptr), MOE_E_ALIAS);
  EXPECT(b.untouched(), 1);
}

}  // namespace

int main() {
  sizes();
  refusals();
  if (g_fail) {
    std::fprintf(stderr, "%d failed\n", g_fail);
    return 1;
  }
  std::printf("all passed\n");
  return 0;
}
