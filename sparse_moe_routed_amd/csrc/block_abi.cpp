// C ABI of the path around the routed experts (the norms before and after a
// block, dispatch, the gradients): host-side validation and dispatch, with
// the rules of moe_abi.cpp -- validation is complete before the first HIP
// call, so a rejected call enqueues nothing and writes nothing.
#include <hip/hip_runtime_api.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "abi_check.h"
#include "moe_internal.h"

namespace moe {

constexpr uint32_t kGateBits = MOE_N_GATE_TOKEN | MOE_N_GATE_FULL;
constexpr uint32_t kNormBits = kGateBits | MOE_N_GATE_SIGMOID | MOE_N_NO_NORM;

static int check_norm(const moe_norm* n) {
  if (!n) return MOE_E_NULL;
  if (n->flags & ~kNormBits) return MOE_E_FLAGS;
  if ((n->flags & kGateBits) == kGateBits) return MOE_E_FLAGS;
  if ((n->flags & MOE_N_GATE_SIGMOID) && !(n->flags & kGateBits)) return MOE_E_FLAGS;
  if (n->act != MOE_DT_F32 && n->act != MOE_DT_BF16) return MOE_E_DTYPE;
  if (n->T < 0 || n->T > 131072 || n->H < 1 || n->H > 65536) return MOE_E_SHAPE;
  // the smallest normal number: a subnormal eps would be flushed to 0
  if (!(n->eps >= FLT_MIN) || !(n->eps <= 0x1p127f)) return MOE_E_VALUE;
  if (!std::isfinite(n->weight_offset) || !std::isfinite(n->residual_scale) ||
      !std::isfinite(n->branch_scale))
    return MOE_E_VALUE;
  return MOE_OK;
}

static size_t norm_act_bytes(const moe_norm& n) { return n.act == MOE_DT_F32 ? 4 : 2; }
static size_t mat_bytes(const moe_norm& n) {
  return static_cast<size_t>(n.T) * n.H * norm_act_bytes(n);
}
static size_t gate_bytes(const moe_norm& n) {
  if (n.flags & MOE_N_GATE_FULL) return mat_bytes(n);
  return n.flags & MOE_N_GATE_TOKEN ? static_cast<size_t>(n.T) * 4 : 0;
}
static size_t part_bytes(const moe_norm& n) {
  return n.T == 0 ? 0
                  : align_up(static_cast<size_t>(norm_bwd_groups(n)) * norm_part_pitch(n.H) * sizeof(float), 256);
}

// A pointer that must be given exactly when `flag` is set.
static int check_flagged(bool flag, const void* p) {
  if (flag) return p ? check_opt_ptr(p) : MOE_E_NULL;
  return p ? MOE_E_FLAGS : MOE_OK;
}

// Weight, gate, residual and next norm of moe_norm_out / moe_combine_norm.
static int check_out_args(const moe_norm& n, const void* w, const void* gate, const void* residual,
                          const void* w_next, const void* out, const void* n_next) {
  int st;
  if ((st = check_ptrs({out}))) return st;
  if ((st = check_flagged(!(n.flags & MOE_N_NO_NORM), w))) return st;
  if ((st = check_flagged((n.flags & kGateBits) != 0, gate))) return st;
  if ((w_next == nullptr) != (n_next == nullptr)) return MOE_E_NULL;
  if ((st = check_opt_ptr(residual)) || (st = check_opt_ptr(w_next)) ||
      (st = check_opt_ptr(n_next)))
    return st;
  return MOE_OK;
}

// dw of an empty batch is a sum over nothing: zeros.
static int empty_dw(const moe_norm& n, float* dw, hipStream_t stream) {
  if (!dw) return MOE_OK;
  if (!aligned16(dw)) return MOE_E_ALIGN;
  (void)hipGetLastError();
  NormBwd a{};
  a.dw = dw;
  return device_status(launch_norm_bwd(n, a, stream));
}

static int check_part(const moe_norm& n, const float* dw, const void* ws, size_t bytes) {
  if (!dw) return MOE_OK;
  if (!ws || bytes < part_bytes(n)) return MOE_E_WORKSPACE;
  return check_opt_ptr(ws);
}

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_norm_workspace_size(const moe_norm* norm) {
  return check_norm(norm) == MOE_OK ? part_bytes(*norm) : 0;
}

int moe_norm_in(const moe_norm* norm, const void* x, const void* w, void* n, hipStream_t stream) {
  int st = check_norm(norm);
  if (st) return st;
  if (norm->flags) return MOE_E_FLAGS;
  if (norm->T == 0) return MOE_OK;
  if ((st = check_ptrs({x, w, n}))) return st;
  const Span outs[] = {{n, mat_bytes(*norm)}};
  const Span ins[] = {{x, mat_bytes(*norm)}, {w, norm->H * norm_act_bytes(*norm)}};
  if (any_alias(outs, 1, ins, 2)) return MOE_E_ALIAS;
  (void)hipGetLastError();
  NormFwd a{};
  a.z = x;
  a.w = w;
  a.out = n;
  moe_norm plain = *norm;
  plain.residual_scale = plain.branch_scale = 1.f;
  return device_status(launch_norm_fwd(plain, a, stream));
}

int moe_norm_in_backward(const moe_norm* norm, const void* dn, const void* x, const void* w,
                         const void* dres, void* dx, float* dw, void* workspace,
                         size_t workspace_bytes, hipStream_t stream) {
  int st = check_norm(norm);
  if (st) return st;
  if (norm->flags) return MOE_E_FLAGS;
  if (norm->T == 0) return empty_dw(*norm, dw, stream);
  if ((st = check_ptrs({dn, x, w, dx}))) return st;
  if ((st = check_opt_ptr(dres)) || (st = check_opt_ptr(dw))) return st;
  if ((st = check_part(*norm, dw, workspace, workspace_bytes))) return st;
  const size_t m = mat_bytes(*norm);
  const Span outs[] = {{dx, m},
                       {dw, dw ? norm->H * sizeof(float) : 0},
                       {workspace, dw ? part_bytes(*norm) : 0}};
  const Span ins[] = {{dn, m}, {x, m}, {w, norm->H * norm_act_bytes(*norm)}, {dres, dres ? m : 0}};
  if (any_alias(outs, 3, ins, 4)) return MOE_E_ALIAS;
  (void)hipGetLastError();
  NormBwd a{};
  a.dout = dn;
  a.z = x;
  a.w = w;
  a.dres = dres;
  a.dz = dx;
  a.dw = dw;
  a.part = static_cast<float*>(workspace);
  moe_norm plain = *norm;
  plain.branch_scale = 1.f;
  return device_status(launch_norm_bwd(plain, a, stream));
}

int moe_norm_out(const moe_norm* norm, const void* z, const void* w, const void* gate,
                 const void* residual, const void* w_next, void* out, void* n_next,
                 hipStream_t stream) {
  int st = check_norm(norm);
  if (st) return st;
  if (norm->T == 0) return MOE_OK;
  if ((st = check_ptrs({z}))) return st;
  if ((st = check_out_args(*norm, w, gate, residual, w_next, out, n_next))) return st;
  const size_t m = mat_bytes(*norm), row = norm->H * norm_act_bytes(*norm);
  const Span outs[] = {{out, m}, {n_next, n_next ? m : 0}};
  const Span ins[] = {{z, m},
                      {w, w ? row : 0},
                      {gate, gate_bytes(*norm)},
                      {residual, residual ? m : 0},
                      {w_next, w_next ? row : 0}};
  if (any_alias(outs, 2, ins, 5)) return MOE_E_ALIAS;
  (void)hipGetLastError();
  NormFwd a{};
  a.z = z;
  a.w = w;
  a.gate = gate;
  a.residual = residual;
  a.w_next = w_next;
  a.out = out;
  a.n_next = n_next;
  return device_status(launch_norm_fwd(*norm, a, stream));
}

int moe_norm_out_backward(const moe_norm* norm, const void* dout, const void* z, const void* w,
                          const void* gate, void* dz, void* dgate, float* dw, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
  int st = check_norm(norm);
  if (st) return st;
  const bool gated = (norm->flags & kGateBits) != 0, normed = !(norm->flags & MOE_N_NO_NORM);
  if ((!normed && dw) || (!gated && dgate)) return MOE_E_FLAGS;
  if (norm->T == 0) return empty_dw(*norm, dw, stream);
  if ((st = check_ptrs({dout, dz}))) return st;
  if ((normed || dgate) && !z) return MOE_E_NULL;   // else nothing reads it
  if ((st = check_opt_ptr(z))) return st;
  if ((st = check_flagged(normed, w)) || (st = check_flagged(gated, gate))) return st;
  if ((st = check_opt_ptr(dgate)) || (st = check_opt_ptr(dw))) return st;
  if ((st = check_part(*norm, dw, workspace, workspace_bytes))) return st;
  const size_t m = mat_bytes(*norm);
  const Span outs[] = {{dz, m},
                       {dgate, dgate ? gate_bytes(*norm) : 0},
                       {dw, dw ? norm->H * sizeof(float) : 0},
                       {workspace, dw ? part_bytes(*norm) : 0}};
  const Span ins[] = {{dout, m},
                      {z, m},
                      {w, w ? norm->H * norm_act_bytes(*norm) : 0},
                      {gate, gate_bytes(*norm)}};
  if (any_alias(outs, 4, ins, 4)) return MOE_E_ALIAS;
  (void)hipGetLastError();
  NormBwd a{};
  a.dout = dout;
  a.z = z;
  a.w = w;
  a.gate = gate;
  a.dz = dz;
  a.dgate = dgate;
  a.dw = dw;
  a.part = static_cast<float*>(workspace);
  return device_status(launch_norm_bwd(*norm, a, stream));
}

int moe_combine_norm(const moe_shape* shape, const moe_norm* norm, const void* y,
                     const int32_t* pair_row, const float* topk_w, const void* w,
                     const void* gate, const void* residual, const void* w_next, void* z,
                     void* out, void* n_next, hipStream_t stream) {
  int st = check_shape(shape);
  if (st) return st;
  if ((st = check_norm(norm))) return st;
  const moe_shape& s = *shape;
  if (norm->T != s.T || norm->H != s.H) return MOE_E_SHAPE;
  if (norm->act != s.act) return MOE_E_DTYPE;
  if (s.T == 0) return MOE_OK;
  if ((st = check_ptrs({y, pair_row, topk_w}))) return st;
  if ((st = check_out_args(*norm, w, gate, residual, w_next, out, n_next))) return st;
  if ((st = check_opt_ptr(z))) return st;
  const size_t m = mat_bytes(*norm), row = norm->H * norm_act_bytes(*norm);
  const size_t P = static_cast<size_t>(s.T) * s.top_k;
  const Span outs[] = {{out, m}, {n_next, n_next ? m : 0}, {z, z ? m : 0}};
  const Span ins[] = {{y, P * row},
                      {pair_row, P * 4},
                      {topk_w, P * 4},
                      {w, w ? row : 0},
                      {gate, gate_bytes(*norm)},
                      {residual, residual ? m : 0},
                      {w_next, w_next ? row : 0}};
  if (any_alias(outs, 3, ins, 7)) return MOE_E_ALIAS;
  (void)hipGetLastError();
  NormFwd a{};
  a.y = y;
  a.pair_row = pair_row;
  a.topk_w = topk_w;
  a.k = s.top_k;
  a.w = w;
  a.gate = gate;
  a.residual = residual;
  a.w_next = w_next;
  a.z_out = z;
  a.out = out;
  a.n_next = n_next;
  return device_status(launch_norm_fwd(*norm, a, stream));
}

int moe_dispatch(const moe_shape* shape, const void* x, const int32_t* pair_row,
                 const float* topk_w, void* rows, hipStream_t stream) {
  int st = check_shape(shape);
  if (st) return st;
  const moe_shape& s = *shape;
  if (s.T == 0) return MOE_OK;
  if ((st = check_ptrs({x, pair_row, rows})) || (st = check_opt_ptr(topk_w))) return st;
  const size_t P = static_cast<size_t>(s.T) * s.top_k, row = s.H * act_bytes(s);
  const Span outs[] = {{rows, P * row}};
  const Span ins[] = {{x, s.T * row}, {pair_row, P * 4}, {topk_w, topk_w ? P * 4 : 0}};
  if (any_alias(outs, 1, ins, 3)) return MOE_E_ALIAS;
  (void)hipGetLastError();
  return device_status(launch_dispatch(s, x, pair_row, topk_w, rows, stream));
}

int moe_dispatch_backward(const moe_shape* shape, const void* drows, const int32_t* pair_row,
                          const float* topk_w, const void* x, const void* dx_in, void* dx,
                          float* dw, hipStream_t stream) {
  int st = check_shape(shape);
  if (st) return st;
  const moe_shape& s = *shape;
  if (s.T == 0) return MOE_OK;
  if ((st = check_ptrs({drows, pair_row, dx}))) return st;
  if (dw && (st = check_ptrs({topk_w, x}))) return st;
  if ((st = check_opt_ptr(topk_w)) || (st = check_opt_ptr(x)) || (st = check_opt_ptr(dx_in)) ||
      (st = check_opt_ptr(dw)))
    return st;
  const size_t P = static_cast<size_t>(s.T) * s.top_k, row = s.H * act_bytes(s), m = s.T * row;
  const Span outs[] = {{dx, m}, {dw, dw ? P * 4 : 0}};
  const Span ins[] = {{drows, P * row},
                      {pair_row, P * 4},
                      {topk_w, topk_w ? P * 4 : 0},
                      {x, x ? m : 0},
                      {dx_in, dx_in ? m : 0}};
  if (any_alias(outs, 2, ins, 5)) return MOE_E_ALIAS;
  (void)hipGetLastError();
  return device_status(launch_dispatch_bwd(s, drows, pair_row, topk_w, x, dx_in, dx, dw, stream));
}

int moe_combine_backward(const moe_shape* shape, const void* dout, const void* y,
                         const int32_t* pair_row, const float* topk_w, void* dy, float* dw,
                         hipStream_t stream) {
  int st = check_shape(shape);
  if (st) return st;
  const moe_shape& s = *shape;
  if (s.T == 0) return MOE_OK;
  if ((st = check_ptrs({dout, pair_row, topk_w, dy}))) return st;
  if (dw && (st = check_ptrs({y}))) return st;
  if ((st = check_opt_ptr(y)) || (st = check_opt_ptr(dw))) return st;
  const size_t P = static_cast<size_t>(s.T) * s.top_k, row = s.H * act_bytes(s);
  const Span outs[] = {{dy, P * row}, {dw, dw ? P * 4 : 0}};
  const Span ins[] = {{dout, s.T * row}, {y, y ? P * row : 0}, {pair_row, P * 4}, {topk_w, P * 4}};
  if (any_alias(outs, 2, ins, 4)) return MOE_E_ALIAS;
  (void)hipGetLastError();
  return device_status(launch_combine_bwd(s, dout, y, pair_row, topk_w, dy, dw, stream));
}

int moe_route_backward(const moe_shape* shape, const int32_t* topk_ids, const float* topk_w,
                       const float* dw, float* dlogits, hipStream_t stream) {
  int st = check_shape(shape);
  if (st) return st;
  const moe_shape& s = *shape;
  if (s.T == 0) return MOE_OK;
  if ((st = check_ptrs({topk_ids, topk_w, dw, dlogits}))) return st;
  const size_t P = static_cast<size_t>(s.T) * s.top_k;
  const Span outs[] = {{dlogits, static_cast<size_t>(s.T) * s.E * 4}};
  const Span ins[] = {{topk_ids, P * 4}, {topk_w, P * 4}, {dw, P * 4}};
  if (any_alias(outs, 1, ins, 3)) return MOE_E_ALIAS;
  (void)hipGetLastError();
  return device_status(launch_route_bwd(s, topk_ids, topk_w, dw, dlogits, stream));
}

}  // extern "C"
