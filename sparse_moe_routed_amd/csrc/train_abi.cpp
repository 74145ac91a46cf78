// C ABI of the training of the routed experts: host-side validation and
// dispatch, with the rules of moe_abi.cpp -- validation is complete before the
// first HIP call, so a rejected call enqueues nothing and writes nothing.
#include <hip/hip_runtime_api.h>

#include <cstdint>

#include "abi_check.h"
#include "moe_internal.h"

namespace moe {

static size_t pairs(const moe_shape& s) { return static_cast<size_t>(s.T) * s.top_k; }

// Shape of the two products: dense row-major expert weights.
static int check_train_shape(const moe_shape* shape, TrainPlan* pl) {
  const int st = check_shape(shape);
  if (st) return st;
  if (shape->wfmt != MOE_WF_DENSE) return MOE_E_FORMAT;
  if (shape->flags & MOE_F_TILED_WEIGHTS) return MOE_E_FLAGS;
  make_train_plan(*shape, pl);
  return train_fits(*shape, *pl) ? MOE_OK : MOE_E_LIMIT;
}

static int check_rows(const moe_perm* pm) {
  return pm ? check_ptrs({pm->offsets, pm->sorted_pair}) : MOE_E_NULL;
}

static int check_saved(const moe_saved* sv) {
  if (!sv) return MOE_E_NULL;
  if (const int st = check_ptrs({sv->g, sv->u})) return st;
  if ((sv->g_scale == nullptr) != (sv->u_scale == nullptr)) return MOE_E_NULL;
  const int st = check_opt_ptr(sv->g_scale);
  return st ? st : check_opt_ptr(sv->u_scale);
}

static bool scaled(const moe_experts& ex) {
  return ex.gate_scale || ex.up_scale || ex.down_scale;
}

static int check_train_ws(const TrainPlan& pl, const void* ws, size_t bytes) {
  if (!ws || bytes < pl.total) return MOE_E_WORKSPACE;
  return check_opt_ptr(ws);
}

static size_t weight_bytes(const moe_shape& s) {
  return static_cast<size_t>(s.E) * s.I * s.H * act_bytes(s);
}

static void saved_spans(const moe_shape& s, const moe_saved& sv, Span* out /*[4]*/) {
  const size_t n = pairs(s) * s.I, m = sv.g_scale ? n : n * act_bytes(s);
  out[0] = {sv.g, m};
  out[1] = {sv.u, m};
  out[2] = {sv.g_scale, sv.g_scale ? n / 32 : 0};
  out[3] = {sv.u_scale, sv.u_scale ? n / 32 : 0};
}

static int check_matrix8(int32_t act, int64_t rows, int64_t cols) {
  if (act != MOE_DT_F32 && act != MOE_DT_BF16) return MOE_E_DTYPE;
  if (rows < 0 || cols < 32 || cols % 32) return MOE_E_SHAPE;
  return rows > (int64_t{1} << 40) / cols ? MOE_E_LIMIT : MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_train_workspace_size(const moe_shape* shape) {
  if (check_shape(shape) != MOE_OK) return 0;
  TrainPlan pl;
  make_train_plan(*shape, &pl);
  return pl.total;
}

int moe_save8(int32_t act, int64_t rows, int64_t cols, const void* v, int8_t* codes,
              uint8_t* scales, hipStream_t stream) {
  int st = check_matrix8(act, rows, cols);
  if (st) return st;
  if (rows == 0) return MOE_OK;
  if ((st = check_ptrs({v, codes, scales}))) return st;
  const bool f32 = act == MOE_DT_F32;
  const size_t n = static_cast<size_t>(rows) * cols;
  const Span outs[] = {{codes, n}, {scales, n / 32}};
  const Span ins[] = {{v, n * (f32 ? 4 : 2)}};
  if (any_alias(outs, 2, ins, 1)) return MOE_E_ALIAS;
  (void)hipGetLastError();
  return device_status(launch_save8(f32, n, v, codes, scales, stream));
}

int moe_restore8(int32_t act, int64_t rows, int64_t cols, const int8_t* codes,
                 const uint8_t* scales, void* v, hipStream_t stream) {
  int st = check_matrix8(act, rows, cols);
  if (st) return st;
  if (rows == 0) return MOE_OK;
  if ((st = check_ptrs({codes, scales, v}))) return st;
  const bool f32 = act == MOE_DT_F32;
  const size_t n = static_cast<size_t>(rows) * cols;
  const Span outs[] = {{v, n * (f32 ? 4 : 2)}};
  const Span ins[] = {{codes, n}, {scales, n / 32}};
  if (any_alias(outs, 1, ins, 2)) return MOE_E_ALIAS;
  (void)hipGetLastError();
  return device_status(launch_restore8(f32, n, codes, scales, v, stream));
}

int moe_ffn_gate_up_save(const moe_shape* shape, const void* x, const moe_experts* experts,
                         const moe_perm* perm, const moe_saved* saved, void* h, void* workspace,
                         size_t workspace_bytes, hipStream_t stream) {
  TrainPlan pl;
  int st = check_train_shape(shape, &pl);
  if (st) return st;
  const moe_shape& s = *shape;
  if (s.T == 0) return MOE_OK;
  if ((st = check_ptrs({x, h}))) return st;
  if (!experts) return MOE_E_NULL;
  if ((st = check_ptrs({experts->gate, experts->up}))) return st;
  if (scaled(*experts)) return MOE_E_FORMAT;
  if ((st = check_rows(perm)) || (st = check_saved(saved))) return st;
  if ((st = check_train_ws(pl, workspace, workspace_bytes))) return st;
  const size_t a = act_bytes(s), P = pairs(s);
  Span outs[6] = {{h, P * s.I * a}, {workspace, pl.total}};
  saved_spans(s, *saved, outs + 2);
  const Span ins[] = {{x, static_cast<size_t>(s.T) * s.H * a},
                      {experts->gate, weight_bytes(s)},
                      {experts->up, weight_bytes(s)},
                      {perm->offsets, (s.E + 1) * 4u},
                      {perm->sorted_pair, P * 4}};
  if (any_alias(outs, 6, ins, 5)) return MOE_E_ALIAS;
  (void)hipGetLastError();
  return device_status(launch_gate_up_save(s, pl, x, *experts, *perm, *saved, h, workspace, stream));
}

int moe_ffn_backward(const moe_shape* shape, const void* dy, const void* x,
                     const uint8_t* x_scale, const moe_saved* saved, const moe_experts* experts,
                     const moe_perm* perm, void* drows, const moe_experts* dexperts,
                     void* workspace, size_t workspace_bytes, hipStream_t stream) {
  TrainPlan pl;
  int st = check_train_shape(shape, &pl);
  if (st) return st;
  const moe_shape& s = *shape;
  if (!drows && !dexperts) return MOE_E_NULL;
  if (dexperts) {
    if ((st = check_ptrs({dexperts->gate, dexperts->up, dexperts->down}))) return st;
    if (scaled(*dexperts)) return MOE_E_FORMAT;
  }
  const size_t a = act_bytes(s), P = pairs(s), m = P * s.H * a, w = weight_bytes(s);
  Span outs[5] = {};
  if (dexperts) {
    outs[0] = {dexperts->gate, w};
    outs[1] = {dexperts->up, w};
    outs[2] = {dexperts->down, w};
  }
  if (s.T == 0) {
    if (!dexperts) return MOE_OK;
    if (any_alias(outs, 3, nullptr, 0)) return MOE_E_ALIAS;
    (void)hipGetLastError();
    return device_status(launch_ffn_backward(s, pl, nullptr, nullptr, nullptr, nullptr,
                                             moe_experts{}, nullptr, nullptr, dexperts, nullptr,
                                             stream));
  }
  if (!dy || (dexperts && !x)) return MOE_E_NULL;
  if ((st = check_ptrs({dy})) || (st = check_opt_ptr(x)) || (st = check_opt_ptr(x_scale)) ||
      (st = check_opt_ptr(drows)))
    return st;
  if ((st = check_saved(saved))) return st;
  if (!experts) return MOE_E_NULL;
  if ((st = check_ptrs({experts->gate, experts->up, experts->down}))) return st;
  if (scaled(*experts)) return MOE_E_FORMAT;
  if ((st = check_rows(perm))) return st;
  if ((st = check_train_ws(pl, workspace, workspace_bytes))) return st;
  outs[3] = {drows, drows ? m : 0};
  outs[4] = {workspace, pl.total};
  const size_t n = static_cast<size_t>(s.T) * s.H;
  Span ins[12] = {{dy, m},
                  {x, x ? n * (x_scale ? 1 : a) : 0},
                  {x_scale, x_scale ? n / 32 : 0},
                  {experts->gate, w},
                  {experts->up, w},
                  {experts->down, w},
                  {perm->offsets, (s.E + 1) * 4u},
                  {perm->sorted_pair, P * 4}};
  saved_spans(s, *saved, ins + 8);
  if (any_alias(outs, 5, ins, 12)) return MOE_E_ALIAS;
  (void)hipGetLastError();
  return device_status(launch_ffn_backward(s, pl, dy, x, x_scale, saved, *experts, perm, drows,
                                           dexperts, workspace, stream));
}

int moe_router_backward(const moe_shape* shape, const int32_t* topk_ids, const float* topk_w,
                        const float* dw, const void* x, const void* w_router, const moe_perm* perm,
                        const void* dx_in, void* dx, float* dw_router, float* dbias,
                        void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int st = check_shape(shape);
  if (st) return st;
  const moe_shape& s = *shape;
  if (!dx && !dw_router && !dbias) return MOE_E_NULL;
  if ((st = check_opt_ptr(dx)) || (st = check_opt_ptr(dw_router)) || (st = check_opt_ptr(dbias)))
    return st;
  const size_t a = act_bytes(s), P = pairs(s), m = static_cast<size_t>(s.T) * s.H * a;
  const size_t we = static_cast<size_t>(s.E) * s.H;
  TrainPlan pl;
  make_train_plan(s, &pl);
  RouterBwd r{};
  r.dw_router = dw_router;
  r.dbias = dbias;
  const bool sums = dw_router || dbias;
  const Span outs[] = {{dx, dx ? m : 0},
                       {dw_router, dw_router ? we * 4 : 0},
                       {dbias, dbias ? s.E * 4u : 0},
                       {workspace, workspace && s.T ? pl.total : 0}};
  if (s.T == 0) {
    if (!sums) return MOE_OK;
    if (any_alias(outs, 3, nullptr, 0)) return MOE_E_ALIAS;
    (void)hipGetLastError();
    return device_status(launch_router_bwd(s, r, stream));
  }
  if ((st = check_ptrs({topk_ids, topk_w, dw}))) return st;
  if ((dx && !w_router) || (dw_router && !x)) return MOE_E_NULL;
  if ((st = check_opt_ptr(x)) || (st = check_opt_ptr(w_router)) || (st = check_opt_ptr(dx_in)))
    return st;
  if (sums) {
    if ((st = check_rows(perm))) return st;
    r.offsets = perm->offsets;
    r.sorted_pair = perm->sorted_pair;
  }
  if ((st = check_train_ws(pl, workspace, workspace_bytes))) return st;
  const Span ins[] = {{topk_ids, P * 4},
                      {topk_w, P * 4},
                      {dw, P * 4},
                      {x, x ? m : 0},
                      {w_router, w_router ? we * a : 0},
                      {dx_in, dx_in ? m : 0},
                      {r.offsets, sums ? (s.E + 1) * 4u : 0},
                      {r.sorted_pair, sums ? P * 4 : 0}};
  if (any_alias(outs, 4, ins, 8)) return MOE_E_ALIAS;
  r.ids = topk_ids;
  r.w = topk_w;
  r.dw = dw;
  r.x = x;
  r.w_router = w_router;
  r.dx_in = dx_in;
  r.dx = dx;
  r.dl = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.dl_off);
  (void)hipGetLastError();
  return device_status(launch_router_bwd(s, r, stream));
}

}  // extern "C"
