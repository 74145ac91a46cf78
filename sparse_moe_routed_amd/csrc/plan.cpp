// Host-side launch planning shared by the C-ABI layer and the launchers:
// which permutation path a shape takes, how the router's H reduction is cut,
// how many fused-FFN slices and route-locality values a shape has.  Plain
// C++ with no device code, so the validation layer builds and runs without
// a GPU.
#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "moe_internal.h"

namespace moe {

// The single-workgroup permutation keeps a token bitmap and its prefix
// counts per expert in LDS (2 words per expert and 32 tokens).
bool permute_single_pass(const moe_shape& s) {
  return static_cast<size_t>(s.E) * ((s.T + 31) / 32) * 2 * sizeof(uint32_t) <= 48 * 1024;
}

int permute_chunks(const moe_shape& s) { return (s.T + kChunkTok - 1) / kChunkTok; }

bool permute_w1_ok(const moe_shape& s) { return s.T <= 32 && s.E <= 1024; }

int router_parts(int H) {
  const int chunks = H / 32;
  int best = 1;
  for (int d = 1; d <= kRouterMaxParts; ++d)
    if (chunks % d == 0) best = d;
  return best;
}

int router_groups(int H) { return (router_parts(H) + kRouterGroup - 1) / kRouterGroup; }

// One workgroup per group of parts multiplies the parallelism of the router
// by the group count (512 tokens: 3.7 us less per layer); at 4096 tokens the
// float64 group sums (groups * T * E * 8 bytes = 64 MB) cost more than the
// parallelism saves (+13 us), so larger batches let the LDS kernel finish
// the sums.
bool router_gsum(const moe_shape& s) { return s.act == MOE_DT_BF16 && s.T <= kRouterGsumMaxT; }

int fused_slices(const moe_shape& s) { return s.I / kFusedCols; }

// 128-row tiles: the bf16 LDS-staged gate/up kernel at 8 token blocks (two
// 16-row blocks of gate and of up per wave; 256 VGPRs with the token
// fragments read one at a time), down on the tiles' two 64-row halves.  At
// 32768 tokens gate/up went 2530 -> 2200 us against 64-row tiles.
bool tiles128_ok(const moe_shape& s) {
  return s.act == MOE_DT_BF16 && s.wfmt == MOE_WF_DENSE && (s.flags & MOE_F_TILED_WEIGHTS) &&
         s.I % 128 == 0;
}

int norm_pack_lanes(int chunks) { return chunks <= 8 ? 8 : chunks <= 16 ? 16 : chunks <= 32 ? 32 : 64; }

// A wave per row (up to 5 16-byte chunks per lane, with their column sums in
// registers) once there are enough rows; few rows finish sooner with a
// workgroup each, and longer rows need one.  2560 bf16, with dw in
// two launches: 1 row 8.5 us (wave) against 4.8 (workgroup), 512 rows 11.1 /
// 9.5, 4096 rows 21.7 / 22.7, 32768 rows 98 / 122; 256 bf16: 2048 rows 6.6 /
// 7.7.
// Rows of at most 32 chunks share a wave.
int norm_bwd_lanes(const moe_norm& n) {
  const int vec = n.act == MOE_DT_BF16 ? 8 : 4, chunks = (n.H + vec - 1) / vec;
  if (n.T < 2048 || chunks > 320) return 0;
  return norm_pack_lanes(chunks);
}

// Four waves, two per SIMD at 512 workgroups; eight where a row is one chunk
// per lane and each wave still gets four rows or more.  With the residual
// path, four against eight: 131072 x 64 bf16 18.5 / 16.9 us, 32768 x 256
// 18.5 / 17.2, 32768 x 384 28.1 / 24.8, 32768 x 333 67 / 44; with fewer rows
// 8192 x 256 8.2 / 9.0, with two chunks per lane 16384 x 1024 28.3 / 29.7.
int norm_bwd_waves(const moe_norm& n) {
  const int vec = n.act == MOE_DT_BF16 ? 8 : 4, lanes = norm_bwd_lanes(n);
  return lanes && n.H <= 64 * vec && n.T / (64 / lanes) >= 16384 ? 8 : 4;
}

// Workgroups of the norm gradient: each leaves one row of column sums, which
// the second launch reads back.  Two per CU; a row each up to 256 rows, then
// two rows or more (512 rows of 2560 bf16: 256 workgroups 8.4 us, 512 9.3;
// 7168 bf16 14.1 / 16.5; at 1536 rows 512 workgroups are ahead, 13.6 / 15.7).
int norm_bwd_groups(const moe_norm& n) {
  if (const int lanes = norm_bwd_lanes(n)) {
    const int rows = norm_bwd_waves(n) * 64 / lanes;
    return std::min((n.T + rows - 1) / rows, 512);
  }
  return std::min(std::max(std::min(n.T, 256), n.T / 2), 512);
}

int locality_blocks(int T) {
  int n = 0;
  for (int B = 1; B <= kMaxLocalityBlock; ++B) n += (T + B - 1) / B;
  return n;
}

}  // namespace moe
