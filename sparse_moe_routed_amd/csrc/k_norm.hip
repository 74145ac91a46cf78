// The norms around a block: norm before it, and norm, gate, residual scale and
// next norm after it, with their gradients (formulas: include/moe.h).
//
// One workgroup per row, element by element, every pass from memory.
#include <algorithm>

#include "moe_internal.h"
#include "row_device.h"

namespace moe {

struct FwdArgs {
  NormFwd a;
  moe_norm n;
  int P;
};

// z[t][h] of the row: the matrix, or the combine of the token's slots
template <class A, bool COMBINE>
__device__ __forceinline__ float branch(const FwdArgs& p, size_t t, int h) {
  typedef typename A::T E;
  if constexpr (!COMBINE) return A::get(static_cast<const E*>(p.a.z)[t * p.n.H + h]);
  float z = 0.f;
  for (int j = 0; j < p.a.k; ++j) {
    const int r = p.a.pair_row[t * p.a.k + j];
    if (r < 0 || r >= p.P) continue;
    z = fmaf(p.a.topk_w[t * p.a.k + j],
             A::get(static_cast<const E*>(p.a.y)[static_cast<size_t>(r) * p.n.H + h]), z);
  }
  return z;
}

template <class A, bool COMBINE>
__global__ __launch_bounds__(256) void k_norm_fwd(FwdArgs p) {
  typedef typename A::T E;
  __shared__ float red[2][4];
  const size_t t = blockIdx.x;
  const int H = p.n.H;
  const bool normed = !(p.n.flags & MOE_N_NO_NORM);
  float rs = 1.f;
  if (normed) {
    float ss = 0.f;
    for (int h = threadIdx.x; h < H; h += 256) {
      const float z = branch<A, COMBINE>(p, t, h);
      ss = fmaf(z, z, ss);
    }
    rs = rsqrtf(row_sum<256>(ss, red[0]) / H + p.n.eps);
  }
  auto value = [&](int h) {
    float v = branch<A, COMBINE>(p, t, h);
    if (normed) v = v * rs * (A::get(static_cast<const E*>(p.a.w)[h]) + p.n.weight_offset);
    if (p.n.flags & (MOE_N_GATE_TOKEN | MOE_N_GATE_FULL)) {
      float g = p.n.flags & MOE_N_GATE_TOKEN ? static_cast<const float*>(p.a.gate)[t]
                                             : A::get(static_cast<const E*>(p.a.gate)[t * H + h]);
      if (p.n.flags & MOE_N_GATE_SIGMOID) g = sigmoid(g);
      v *= g;
    }
    v *= p.n.branch_scale;
    if (p.a.residual)
      v = fmaf(p.n.residual_scale, A::get(static_cast<const E*>(p.a.residual)[t * H + h]), v);
    return v;
  };
  float ss = 0.f;
  for (int h = threadIdx.x; h < H; h += 256) {
    const float v = value(h);
    static_cast<E*>(p.a.out)[t * H + h] = A::put(v);
    if (p.a.z_out) static_cast<E*>(p.a.z_out)[t * H + h] = A::put(branch<A, COMBINE>(p, t, h));
    ss = fmaf(v, v, ss);
  }
  if (!p.a.n_next) return;
  const float rn = rsqrtf(row_sum<256>(ss, red[1]) / H + p.n.eps);
  for (int h = threadIdx.x; h < H; h += 256)
    static_cast<E*>(p.a.n_next)[t * H + h] =
        A::put(value(h) * rn * (A::get(static_cast<const E*>(p.a.w_next)[h]) + p.n.weight_offset));
}

hipError_t launch_norm_fwd(const moe_norm& n, const NormFwd& a, hipStream_t st) {
  const FwdArgs p{a, n, n.T * a.k};
  const bool bf = n.act == MOE_DT_BF16;
  auto kern = a.y ? (bf ? k_norm_fwd<RowBf16, true> : k_norm_fwd<RowF32, true>)
                  : (bf ? k_norm_fwd<RowBf16, false> : k_norm_fwd<RowF32, false>);
  hipLaunchKernelGGL(kern, dim3(n.T), dim3(256), 0, st, p);
  return hipGetLastError();
}

struct BwdArgs {
  NormBwd a;
  moe_norm n;
};

// Workgroup g takes rows g, g + G, ...; its column sums of dw stay in its row
// of `part`, which only its own threads touch.
template <class A>
__global__ __launch_bounds__(256) void k_norm_bwd(BwdArgs p) {
  typedef typename A::T E;
  __shared__ float red[2][2][4];
  const int H = p.n.H;
  const bool normed = !(p.n.flags & MOE_N_NO_NORM);
  const bool sig = p.n.flags & MOE_N_GATE_SIGMOID;
  const E* dout = static_cast<const E*>(p.a.dout);
  const E* z = static_cast<const E*>(p.a.z);
  const E* w = static_cast<const E*>(p.a.w);
  float* part = p.a.dw ? p.a.part + static_cast<size_t>(blockIdx.x) * H : nullptr;
  int round = 0;
  for (int t = blockIdx.x; t < p.n.T; t += gridDim.x, ++round) {
    const size_t o = static_cast<size_t>(t) * H;
    float gt = 1.f;
    if (p.n.flags & MOE_N_GATE_TOKEN) {
      gt = static_cast<const float*>(p.a.gate)[t];
      if (sig) gt = sigmoid(gt);
    }
    auto gate = [&](int h) {
      if (!(p.n.flags & MOE_N_GATE_FULL)) return gt;
      const float g = A::get(static_cast<const E*>(p.a.gate)[o + h]);
      return sig ? sigmoid(g) : g;
    };
    auto weight = [&](int h) { return normed ? A::get(w[h]) + p.n.weight_offset : 1.f; };
    float ss = 0.f, s1 = 0.f;   // sum z^2, sum G db w z
    for (int h = threadIdx.x; h < H; h += 256) {
      const float zz = A::get(z[o + h]), d = p.n.branch_scale * A::get(dout[o + h]);
      ss = fmaf(zz, zz, ss);
      s1 = fmaf((p.n.flags & MOE_N_GATE_FULL ? gate(h) : 1.f) * d * weight(h), zz, s1);
    }
    ss = row_sum<256>(ss, red[round & 1][0]);
    s1 = row_sum<256>(s1, red[round & 1][1]);
    const float rs = normed ? rsqrtf(ss / H + p.n.eps) : 1.f;
    if (p.n.flags & MOE_N_GATE_TOKEN) {
      if (p.a.dgate && threadIdx.x == 0)
        static_cast<float*>(p.a.dgate)[t] = rs * s1 * (sig ? gt * (1.f - gt) : 1.f);
      s1 *= gt;
    }
    const float c = normed ? rs * s1 / H : 0.f;   // mean(g zh)
    for (int h = threadIdx.x; h < H; h += 256) {
      const float zh = A::get(z[o + h]) * rs, d = p.n.branch_scale * A::get(dout[o + h]);
      const float G = gate(h), wh = weight(h);
      float dz = G * d * wh;
      if (normed) dz = rs * (dz - zh * c);
      if (p.a.dres) dz = fmaf(p.n.residual_scale, A::get(static_cast<const E*>(p.a.dres)[o + h]), dz);
      static_cast<E*>(p.a.dz)[o + h] = A::put(dz);
      if (p.a.dgate && (p.n.flags & MOE_N_GATE_FULL))
        static_cast<E*>(p.a.dgate)[o + h] = A::put(d * zh * wh * (sig ? G * (1.f - G) : 1.f));
      if (part) part[h] = (round ? part[h] : 0.f) + G * d * zh;
    }
  }
}

__global__ __launch_bounds__(256) void k_norm_dw(const float* part, float* dw, int G, int H) {
  const int h = blockIdx.x * 256 + threadIdx.x;
  if (h >= H) return;
  float s = 0.f;
  for (int g = 0; g < G; ++g) s += part[static_cast<size_t>(g) * H + h];
  dw[h] = s;
}

hipError_t launch_norm_bwd(const moe_norm& n, const NormBwd& a, hipStream_t st) {
  const int G = norm_bwd_groups(n);
  const BwdArgs p{a, n};
  if (n.T > 0) {
    auto kern = n.act == MOE_DT_BF16 ? k_norm_bwd<RowBf16> : k_norm_bwd<RowF32>;
    hipLaunchKernelGGL(kern, dim3(G), dim3(256), 0, st, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.dw)
    hipLaunchKernelGGL(k_norm_dw, dim3((n.H + 255) / 256), dim3(256), 0, st, a.part, a.dw, G, n.H);
  return hipGetLastError();
}

}  // namespace moe
