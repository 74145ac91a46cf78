// Host-only validation battery of the entry points around the routed experts
// (block_abi.cpp), built with AddressSanitizer and UndefinedBehaviorSanitizer
// and launchers that abort if reached: every call below must be refused (or
// is an empty batch), reach no launcher and leave its sentinel buffers alone.
// Workspace sizes are computed over the corners of the domain.
#include <cmath>
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

hipError_t launch_norm_fwd(const moe_norm&, const NormFwd&, hipStream_t) { reached("launch_norm_fwd"); }
hipError_t launch_norm_bwd(const moe_norm&, const NormBwd&, hipStream_t) { reached("launch_norm_bwd"); }
hipError_t launch_dispatch(const moe_shape&, const void*, const int32_t*, const float*, void*,
                           hipStream_t) { reached("launch_dispatch"); }
hipError_t launch_dispatch_bwd(const moe_shape&, const void*, const int32_t*, const float*,
                               const void*, const void*, void*, float*, hipStream_t) {
  reached("launch_dispatch_bwd");
}
hipError_t launch_combine_bwd(const moe_shape&, const void*, const void*, const int32_t*,
                              const float*, void*, float*, hipStream_t) { reached("launch_combine_bwd"); }
hipError_t launch_route_bwd(const moe_shape&, const int32_t*, const float*, const float*, float*,
                            hipStream_t) { reached("launch_route_bwd"); }

}  // namespace moe

namespace {

int g_fail = 0;

void expect(int line, int got, int want) {
  if (got == want) return;
  std::fprintf(stderr, "FAIL %s:%d: status %d, want %d\n", __FILE__, line, got, want);
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

moe_norm norm(int T, int H, int act = MOE_DT_BF16, uint32_t flags = 0) {
  return moe_norm{T, H, act, flags, 1e-6f, 0.f, 1.f, 1.f};
}

}  // namespace

int main() {
  std::vector<Buf> b(11, Buf(1 << 14));
  for (Buf& x : b) x = Buf(1 << 14);
  void* p[11];
  for (int i = 0; i < 11; ++i) p[i] = b[i].p;
  const int32_t* ip = reinterpret_cast<const int32_t*>(p[1]);
  const float* fp = reinterpret_cast<const float*>(p[2]);
  float* fo = reinterpret_cast<float*>(p[9]);
  const size_t big = size_t{1} << 40;

  // workspace sizes over the domain's corners
  for (int T : {0, 1, 2, 511, 512, 513, 4096, 131072})
    for (int H : {1, 7, 64, 2560, 65535, 65536})
      for (int act : {0, 1}) {
        const moe_norm n = norm(T, H, act);
        const size_t w = moe_norm_workspace_size(&n);
        EXPECT(T == 0 ? w == 0 : w >= static_cast<size_t>(H) * 4 && w % 256 == 0, 1);
      }

  // descriptors
  const float bad[] = {0.f, -1.f, 1e-40f, std::numeric_limits<float>::quiet_NaN(),
                       std::numeric_limits<float>::infinity()};
  for (float e : bad) {
    moe_norm n = norm(4, 96);
    n.eps = e;
    EXPECT(moe_norm_in(&n, p[0], p[1], p[2], nullptr), MOE_E_VALUE);
    n = norm(4, 96);
    n.branch_scale = std::isfinite(e) ? std::numeric_limits<float>::infinity() : e;
    EXPECT(moe_norm_out(&n, p[0], p[1], nullptr, p[3], p[4], p[5], p[6], nullptr), MOE_E_VALUE);
  }
  for (int T : {INT32_MIN, -1, 131073, INT32_MAX})
    for (int H : {96, INT32_MAX}) {
      const moe_norm n = norm(T, H);
      EXPECT(moe_norm_in(&n, p[0], p[1], p[2], nullptr), MOE_E_SHAPE);
      EXPECT(moe_norm_in_backward(&n, p[0], p[1], p[2], p[3], p[4], fo, p[5], big, nullptr), MOE_E_SHAPE);
      EXPECT(moe_norm_out_backward(&n, p[0], p[1], p[2], nullptr, p[4], nullptr, fo, p[5], big, nullptr),
             MOE_E_SHAPE);
      EXPECT(moe_norm_workspace_size(&n) == 0, 1);
    }
  for (uint32_t f : {16u, 0x80000000u, 3u, 4u, 12u}) {
    const moe_norm n = norm(4, 96, MOE_DT_BF16, f);
    EXPECT(moe_norm_out(&n, p[0], p[1], p[2], p[3], p[4], p[5], p[6], nullptr), MOE_E_FLAGS);
  }

  // overlaps at the far end of the largest matrices (addresses only)
  {
    const moe_norm n = norm(131072, 65536, MOE_DT_F32);
    char* base = reinterpret_cast<char*>(uintptr_t{1} << 44);
    const size_t m = size_t{131072} * 65536 * 4;
    EXPECT(moe_norm_in(&n, base, base + 2 * m, base + m - 16, nullptr), MOE_E_ALIAS);
    EXPECT(moe_norm_in_backward(&n, base, base + m, base + 4 * m, nullptr, base + 2 * m - 16, nullptr, nullptr,
                                0, nullptr), MOE_E_ALIAS);
  }
  {
    const moe_shape s{131072, 16256, 1024, 64, 60, MOE_DT_F32, MOE_WF_DENSE, 0};
    char* base = reinterpret_cast<char*>(uintptr_t{1} << 44);
    const size_t m = size_t{131072} * 16256 * 4;
    EXPECT(moe_dispatch(&s, base + 60 * m - 16, ip, nullptr, base, nullptr), MOE_E_LIMIT);
    const moe_shape s2{131072, 16256, 1024, 64, 6, MOE_DT_F32, MOE_WF_DENSE, 0};
    EXPECT(moe_dispatch(&s2, base + 6 * m - 16, ip, nullptr, base, nullptr), MOE_E_ALIAS);
    EXPECT(moe_combine_backward(&s2, base + 20 * m, base, ip, fp, base + 6 * m - 16, nullptr, nullptr),
           MOE_E_ALIAS);
  }

  // workspace, null and empty
  {
    const moe_norm n = norm(4, 96);
    const size_t need = moe_norm_workspace_size(&n);
    EXPECT(moe_norm_in_backward(&n, p[0], p[1], p[2], p[3], p[4], fo, p[5], need - 1, nullptr), MOE_E_WORKSPACE);
    EXPECT(moe_norm_in_backward(&n, p[0], p[1], p[2], p[3], p[4], fo, nullptr, need, nullptr), MOE_E_WORKSPACE);
    EXPECT(moe_norm_in_backward(&n, p[0], p[1], p[2], p[3], p[4], fo, p[9], need, nullptr), MOE_E_ALIAS);
    EXPECT(moe_norm_in(nullptr, p[0], p[1], p[2], nullptr), MOE_E_NULL);
    const moe_norm e = norm(0, 96);
    EXPECT(moe_norm_in_backward(&e, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr),
           MOE_OK);
    EXPECT(moe_norm_in_backward(&e, nullptr, nullptr, nullptr, nullptr, nullptr, fo + 1, nullptr, 0, nullptr),
           MOE_E_ALIGN);
  }
  {
    const moe_shape s{4, 128, 8, 64, 2, MOE_DT_BF16, MOE_WF_DENSE, 0};
    EXPECT(moe_dispatch_backward(&s, p[0], ip, nullptr, p[3], nullptr, p[4], fo, nullptr), MOE_E_NULL);
    EXPECT(moe_dispatch_backward(&s, p[0], ip, fp, nullptr, nullptr, p[4], fo, nullptr), MOE_E_NULL);
    EXPECT(moe_combine_backward(&s, p[0], nullptr, ip, fp, p[4], fo, nullptr), MOE_E_NULL);
    EXPECT(moe_route_backward(&s, ip, fp, fo, fo, nullptr), MOE_E_ALIAS);
    EXPECT(moe_route_backward(nullptr, ip, fp, fp, fo, nullptr), MOE_E_NULL);
  }

  for (const Buf& x : b)
    if (!x.untouched()) {
      std::fprintf(stderr, "FAIL: a sentinel buffer was written\n");
      ++g_fail;
    }
  if (g_fail) return 1;
  std::puts("all passed");
  return 0;
}
