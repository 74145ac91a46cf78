// Internal interface between the C-ABI layer (moe_abi.cpp) and the kernel
// launchers.  Nothing here is exported.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

// Sizes shared by the host planning code (plan.cpp) and the kernels.
constexpr int kChunkTok = 256;          // tokens per chunk of the large-batch permutation
constexpr int kRouterGroup = 4;         // consecutive H parts whose sums are added first
constexpr int kRouterMaxParts = 16;     // parts of the router's H reduction, at most
constexpr int kRouterMaxGroups = kRouterMaxParts / kRouterGroup;
constexpr int kRouterGsumMaxT = 1024;   // group sums finished by the top-k kernel up to here
constexpr int kFusedCols = 64;          // intermediate columns per fused-FFN work item
constexpr int kMaxLocalityBlock = 5;    // route-locality block sizes 1..5

// Launch geometry and workspace layout for one shape.  Every region is
// 256-byte aligned; moe_workspace_size() returns `total`.
struct Plan {
  // router
  size_t logits_off;      // float [T][E] (when the caller passes no logits buffer)
  size_t gsum_off;        // double [router groups][T][E] (bf16 batches up to 1024 tokens)
  // permutation
  int chunks;             // 256-token chunks of the large-batch path (0: one pass)
  size_t chunk_off;       // int32 chunk counts [chunks][E] + chunk bases [chunks][E]
  size_t perm_off;        // int32 counts[E], offsets[E+1], sorted_pair[P],
                          // pair_row[P], active[E], n_active[1]
  // grouped FFN
  int nb;                 // 16-row token groups per tile (rows per tile = 16*nb)
  int max_tiles;          // upper bound on tiles: P/(16 nb) + min(E, P)
  size_t tiles_off;       // int32 [3*max_tiles] (expert, row0, rows) + n_tiles + the
                          // route + permute arrival counter
  size_t h_off;           // act [P][I] SwiGLU intermediate
  size_t y_off;           // act [P][H] expert outputs (moe_layer only)
  // MOE_F_CHECK_FINITE: private results until the status word is clean
  size_t ids_off;         // int32 [P]
  size_t w_off;           // float [P]
  size_t out_off;         // act [T][H] (moe_layer)
  size_t status_off;      // uint32 status word
  // MOE_F_FUSED_FFN: float [I/64][P][H] partial expert outputs
  size_t part_off;
  size_t total;
};

bool make_plan(const moe_shape& s, Plan* p);

// MOE_OK when the shape is in the domain of include/moe.h
int check_shape(const moe_shape* s);

// Supplies the workspace of a validated moe_layer call that received none:
// `need` is the plan's size; on MOE_OK *ws / *ws_bytes describe device
// memory of at least `need` bytes usable on `st`'s device.
typedef int (*ScratchFn)(size_t need, hipStream_t st, void** ws, size_t* ws_bytes);

// moe_layer with an optional scratch supplier (nullptr: the caller's
// workspace); every validation step runs before `scratch` is called.
int layer_call(const moe_shape* shape, const void* x, const void* w_router, const float* router_bias,
               const moe_experts* experts, const void* residual, void* out, int32_t* topk_ids,
               float* topk_w, const moe_perm* perm, void* workspace, size_t workspace_bytes,
               hipStream_t stream, ScratchFn scratch);

struct PermPtrs {
  int32_t *counts, *offsets, *sorted_pair, *pair_row, *active, *n_active;
};

// Launchers: enqueue only, return hipGetLastError().
int router_parts(int H);        // parts of the H reduction (largest divisor of H/32 <= 16)
int router_groups(int H);       // groups of consecutive parts
bool router_gsum(const moe_shape& s);   // router group sums finished by the top-k kernel
hipError_t launch_route(const moe_shape& s, const Plan& pl, const void* x, const void* w_router,
                        const float* bias, int32_t* ids, float* w, float* logits, void* ws,
                        hipStream_t st);
// route + permute in one call: fused (the top-k kernel's last workgroup
// builds the permutation) for bf16 batches of up to 32 tokens, else the two
// launches back to back
bool route_permute_fused(const moe_shape& s);
hipError_t launch_route_permute(const moe_shape& s, const Plan& pl, const void* x,
                                const void* w_router, const float* bias, int32_t* ids, float* w,
                                float* logits, const PermPtrs& pp, int32_t* tiles, void* ws,
                                hipStream_t st);
bool permute_single_pass(const moe_shape& s);
bool permute_w1_ok(const moe_shape& s);   // the 32-token permutation (one bitmap word per expert)
int permute_chunks(const moe_shape& s);
hipError_t launch_permute(const moe_shape& s, const Plan& pl, const int32_t* ids,
                          const PermPtrs& pp, int32_t* tiles /* may be null */, void* ws,
                          hipStream_t st);
hipError_t launch_plan_tiles(const moe_shape& s, const Plan& pl, const PermPtrs& pp,
                             int32_t* tiles, hipStream_t st);
hipError_t launch_gateup(const moe_shape& s, const Plan& pl, const void* x, const moe_experts& ex,
                         const int32_t* sorted_pair, const int32_t* tiles, void* h,
                         hipStream_t st);
hipError_t launch_down(const moe_shape& s, const Plan& pl, const void* h, const moe_experts& ex,
                       const int32_t* tiles, void* y, hipStream_t st);
// 128-row tiles (nb = 8) are planned only for bf16 tiled weights
bool tiles128_ok(const moe_shape& s);
hipError_t launch_ffn(const moe_shape& s, const Plan& pl, const void* x, const moe_experts& ex,
                      const int32_t* sorted_pair, const int32_t* tiles, void* h, void* y,
                      hipStream_t st);
// down then combine (y in `y`): with 16-row tiles of tiled bf16-activation
// weights y goes to pair slots and the combine reads them directly
bool down_pair_order(const moe_shape& s, const Plan& pl);
hipError_t launch_down_combine(const moe_shape& s, const Plan& pl, const void* h,
                               const moe_experts& ex, const int32_t* tiles,
                               const int32_t* sorted_pair, const int32_t* pair_row, const float* w,
                               const void* residual, void* out, void* y, hipStream_t st);
int fused_slices(const moe_shape& s);   // I / 64
hipError_t launch_ffn_fused(const moe_shape& s, const Plan& pl, const void* x,
                            const moe_experts& ex, const int32_t* sorted_pair,
                            const int32_t* tiles, float* part, int wave_tiles, uint64_t* clock,
                            hipStream_t st);
hipError_t launch_reduce_parts(const moe_shape& s, const float* part, void* y, hipStream_t st);
hipError_t launch_combine_parts(const moe_shape& s, const float* part, const int32_t* pair_row,
                                const float* w, const void* residual, void* out, hipStream_t st);
hipError_t launch_tile_experts(const moe_shape& s, const moe_experts& src, const moe_experts& dst,
                               hipStream_t st);
int locality_blocks(int T);   // sum over B = 1..5 of ceil(T / B)
hipError_t launch_route_locality(const moe_shape& s, const int32_t* ids, int32_t* overlap,
                                 int32_t* block_unique, hipStream_t st);
// Per-expert byte pieces of one expert record set (gate, up, down and their
// scales): source and destination bases (device-usable addresses) and bytes
// per expert; a null source skips the piece.
constexpr int kStagePieces = 6;
struct StagePieces {
  const char* src[kStagePieces];
  char* dst[kStagePieces];
  size_t bytes[kStagePieces];
};
hipError_t launch_stage_experts(const moe_shape& s, const StagePieces& pc, const int32_t* active,
                                const int32_t* n_active, hipStream_t st);
hipError_t launch_stream_read(const void* buf, size_t bytes, uint32_t* sink, hipStream_t st);
hipError_t launch_zero_status(uint32_t* status, hipStream_t st);
// sets `bit` in *status if any of the n values (bf16 or float32) is NaN/inf
hipError_t launch_check_finite(const void* src, size_t n, bool bf16, uint32_t bit,
                               uint32_t* status, hipStream_t st);
// Inputs that a call reads once bypass the caches (non-temporal) when they
// could not stay there anyway; smaller ones may have just been written by the
// call before.  Measured on pairs of calls that hand their output on, plain
// against non-temporal loads, 2560 bf16:
//   norm_out then norm_in gradient: matrices of 2.6 MB 8.9 / 9.4 us, 5.2 MB
//   13.7 / 13.7, 7.9 MB 18.3 / 16.6, 21 MB 30.1 / 28.4, 84 MB 110 / 93 (a call
//   has four or five matrices, the L2s hold 32 MB);
//   dispatch, combine gradient, dispatch gradient, top-10: rows of 105 MB
//   79 / 84 us, 157 MB 141 / 120, 210 MB 193 / 157 (two such matrices pass the
//   256 MB cache in front of HBM).
// Outputs are written through the caches at every size here: the next call
// reads them (norm_out then norm_in gradient, 84 MB: 93 us against 100).
constexpr bool streams_matrix(size_t bytes) { return bytes >= size_t{6} << 20; }
constexpr bool streams_slots(size_t bytes) { return bytes >= size_t{128} << 20; }

// The norms around the block.  Forward: z is a matrix, or (y, pair_row,
// topk_w, k given) the combine of a token's slots; norm_in is the forward
// kernel without gate, residual and next norm.
struct NormFwd {
  const void* z;
  const void* y;
  const int32_t* pair_row;
  const float* topk_w;
  int k;
  const void *w, *gate, *residual, *w_next;
  void *z_out, *out, *n_next;
};
struct NormBwd {
  const void *dout, *z, *w, *gate, *dres;
  void *dz, *dgate;
  float *dw, *part;   // part: float [norm_bwd_groups][norm_part_pitch(H)]
};
int norm_pack_lanes(int chunks);          // lanes of a row of that many chunks (8 .. 64)
int norm_bwd_lanes(const moe_norm& n);    // lanes of a row in the gradient, 0: a workgroup
int norm_bwd_waves(const moe_norm& n);    // waves of a gradient workgroup, if a row has lanes
constexpr int norm_part_pitch(int H) { return (H + 7) / 8 * 8; }
int norm_bwd_groups(const moe_norm& n);   // workgroups of the gradient kernel
hipError_t launch_norm_fwd(const moe_norm& n, const NormFwd& a, hipStream_t st);
hipError_t launch_norm_bwd(const moe_norm& n, const NormBwd& a, hipStream_t st);
// token rows in expert order and the gradients of dispatch, combine, route
hipError_t launch_dispatch(const moe_shape& s, const void* x, const int32_t* pair_row,
                           const float* w, void* rows, hipStream_t st);
hipError_t launch_dispatch_bwd(const moe_shape& s, const void* drows, const int32_t* pair_row,
                               const float* w, const void* x, const void* dx_in, void* dx,
                               float* dw, hipStream_t st);
hipError_t launch_combine_bwd(const moe_shape& s, const void* dout, const void* y,
                              const int32_t* pair_row, const float* w, void* dy, float* dw,
                              hipStream_t st);
hipError_t launch_route_bwd(const moe_shape& s, const int32_t* ids, const float* w,
                            const float* dw, float* dlogits, hipStream_t st);
// pair_row == nullptr: y rows in pair order (row t*k + j)
hipError_t launch_combine(const moe_shape& s, const void* y, const int32_t* pair_row,
                          const float* w, const void* residual, void* out, hipStream_t st);

// Training the routed experts (k_train*.hip, k_save8.hip, k_router_bwd.hip).
// How one product over the experts' rows is cut: the tile shape, and into how
// many parts its sum (float32 partial results, joined by another launch).
enum RowShape { kRowsFew = 0, kRowsMany = 1, kRowsWide = 2 };
struct RowCut {
  int shape;   // RowShape
  int parts;
};
constexpr int row_height(int shape) { return shape == kRowsFew ? 32 : shape == kRowsMany ? 128 : 256; }
constexpr int kLookupExperts = 64;   // up to here a wave finds its tile itself
constexpr int kJointBlocks = 512;    // most workgroups of the rows' gradient that share the weight gradients' launch
#ifdef __HIPCC__
#define MOE_BOTH __host__ __device__ inline
#else
#define MOE_BOTH inline
#endif
// Tiles of 256 x 256 take a CU each.  Those that are left when the others have filled
// the 256 CUs `full / 256` times are cut along their sum, so that they fill them once
// more, and another kernel joins them (8192 x 2560 x 5120: dx is 320 tiles, dw 600).
constexpr int kCus = 256, kMostCuts = 4, kTailBytes = 256 * 256 * 4;
struct Tail {
  int full, rest, cut;
  static constexpr bool possible(int stages) { return stages >= 16; }
  MOE_BOTH Tail(int total, int stages) {
    full = total / kCus * kCus;
    rest = total - full;
    cut = 1;
    if (rest > 0 && rest <= kCus / 2) {
      cut = kCus / rest;
      if (cut > kMostCuts) cut = kMostCuts;
      if (cut > stages / 8) cut = stages / 8;
    }
    if (cut < 2) {
      full = total;
      rest = 0;
      cut = 1;
    }
  }
  // Item of a workgroup: consecutive ones go to one XCD (workgroups are dealt to the
  // 8 XCDs in turn).
  MOE_BOTH bool item(int block, int& tile, int& part, int& slot) const {
    int per = (full + 7) / 8, turn = block >> 3, at = (block & 7) * per + turn;
    part = slot = 0;
    tile = at;
    if (turn < per) return at < full;
    turn -= per;
    per = (rest * cut + 7) / 8;
    slot = (block & 7) * per + turn;
    if (turn >= per || slot >= rest * cut) return false;
    tile = full + slot / cut;
    part = slot % cut;
    return true;
  }
};

// Workspace of one shape; the regions of the two products and of the router's
// gradient overlap, as no call uses both.
struct TrainPlan {
  RowCut gate_up, dh, dx;
  int dw_parts;   // parts of an expert's rows in the weight gradients, 0: by 256 x 256 tiles
  bool joint;     // the rows' and the weights' gradients, where both are wanted, are one launch
  // tile lists, by row height 32 or 128 / 256: int32 [3 * most] (expert, row0, rows), then their number
  int most[2];
  size_t tiles_off[2];
  size_t x_off;         // act [T][H], x read back from an 8-bit checkpoint
  size_t dg_off, du_off, h_off;   // act [P][I]
  size_t rows_part_off; // float [parts][P][columns], or the tiles of 256 x 256 that are cut
  size_t dw_part_off;   // float [dw_parts][3][E][I H], or the same
  size_t dl_off;        // router: float [P]
  size_t total;
};
void make_train_plan(const moe_shape& s, TrainPlan* p);
// Whether an expert's rows are about one tile, so that a weight is read about once.
bool read_once(const moe_shape& s, const RowCut& c);
bool train_fits(const moe_shape& s, const TrainPlan& p);   // the limits of the two products

hipError_t launch_save8(bool f32, size_t n, const void* v, int8_t* codes, uint8_t* scales,
                        hipStream_t st);
hipError_t launch_restore8(bool f32, size_t n, const int8_t* codes, const uint8_t* scales, void* v,
                           hipStream_t st);
hipError_t launch_gate_up_save(const moe_shape& s, const TrainPlan& pl, const void* x,
                               const moe_experts& ex, const moe_perm& pm, const moe_saved& sv,
                               void* h, void* ws, hipStream_t st);
hipError_t launch_ffn_backward(const moe_shape& s, const TrainPlan& pl, const void* dy,
                               const void* x, const uint8_t* x_scale, const moe_saved* sv,
                               const moe_experts& ex, const moe_perm* pm, void* drows,
                               const moe_experts* dex, void* ws, hipStream_t st);
struct RouterBwd {
  const int32_t* ids;
  const float *w, *dw;
  const void *x, *w_router, *dx_in;
  const int32_t *offsets, *sorted_pair;
  void* dx;
  float *dw_router, *dbias, *dl;
};
hipError_t launch_router_bwd(const moe_shape& s, const RouterBwd& a, hipStream_t st);

}  // namespace moe
