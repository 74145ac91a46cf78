// Gradient of the router's product.
//
// Only the top_k selected logits of a token have a gradient, so both products
// are sparse: dx gathers top_k rows of w_router per token, dw_router sums the
// tokens of an expert's rows.  4 P H flops against 3 T H a + E H (a + 4) bytes:
// bound by memory and, through the gathers, by the caches.
#include "moe_internal.h"
#include "row_device.h"

namespace moe {

// One workgroup per token: dl of its pairs, then dx.
template <class A>
__global__ __launch_bounds__(256) void k_router_dx(RouterBwd a, int H, int E, int k) {
  typedef typename A::T T;
  constexpr int V = A::VEC;
  __shared__ float dl[1024];
  __shared__ float part[4];
  const size_t p0 = static_cast<size_t>(blockIdx.x) * k;
  float dot = 0.f;
  for (int j = threadIdx.x; j < k; j += 256) dot = fmaf(a.w[p0 + j], a.dw[p0 + j], dot);
  dot = wave_sum_f32(dot);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
  __syncthreads();
  dot = (part[0] + part[1]) + (part[2] + part[3]);
  for (int j = threadIdx.x; j < k; j += 256) {
    const float d = a.w[p0 + j] * (a.dw[p0 + j] - dot);
    dl[j] = d;
    a.dl[p0 + j] = d;
  }
  __syncthreads();
  if (!a.dx) return;
  const T* wr = static_cast<const T*>(a.w_router);
  const size_t row = static_cast<size_t>(blockIdx.x) * H;
  for (int h = threadIdx.x * V; h < H; h += 256 * V) {
    float v[V];
    if (a.dx_in)
      A::unpack(ld16(static_cast<const T*>(a.dx_in) + row + h), v);
    else
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = 0.f;
    for (int j = 0; j < k; ++j) {
      const int e = a.ids[p0 + j];
      if (static_cast<uint32_t>(e) >= static_cast<uint32_t>(E)) continue;
      float r[V];
      A::unpack(ld16(wr + static_cast<size_t>(e) * H + h), r);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = fmaf(dl[j], r[i], v[i]);
    }
    *reinterpret_cast<u32x4_t*>(static_cast<T*>(a.dx) + row + h) = A::pack(v);
  }
}

// One workgroup per expert and 64 V features: four waves share the rows.
template <class A>
__global__ __launch_bounds__(256) void k_router_dw(RouterBwd a, int H, int P, int k) {
  typedef typename A::T T;
  constexpr int V = A::VEC;
  __shared__ float sums[4][64 * V];
  __shared__ float bias[4];
  const int e = blockIdx.x, w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int h = (blockIdx.y * 64 + lane) * V;
  int row0 = 0, rows = 0;
  if (P > 0) {
    row0 = min(max(a.offsets[e], 0), P);
    rows = min(max(a.offsets[e + 1], row0), P) - row0;
  }
  float v[V] = {}, db = 0.f;
  for (int r = w; r < rows; r += 4) {
    const int p = min(max(a.sorted_pair[row0 + r], 0), P - 1);
    const float d = a.dl[p];
    db += d;
    if (a.dw_router && h < H) {
      float x[V];
      A::unpack(ld16(static_cast<const T*>(a.x) + static_cast<size_t>(p / k) * H + h), x);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = fmaf(d, x[i], v[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) sums[w][lane * V + i] = v[i];
  if (lane == 0) bias[w] = db;
  __syncthreads();
  if (a.dw_router)
    for (int i = threadIdx.x; i < 64 * V; i += 256) {
      const int c = blockIdx.y * 64 * V + i;
      if (c < H) a.dw_router[static_cast<size_t>(e) * H + c] = (sums[0][i] + sums[1][i]) + (sums[2][i] + sums[3][i]);
    }
  if (a.dbias && blockIdx.y == 0 && threadIdx.x == 0) a.dbias[e] = (bias[0] + bias[1]) + (bias[2] + bias[3]);
}

template <class A>
static hipError_t run(const moe_shape& s, const RouterBwd& a, hipStream_t st) {
  if (s.T > 0) {
    k_router_dx<A><<<s.T, 256, 0, st>>>(a, s.H, s.E, s.top_k);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  if (a.dw_router || a.dbias)
    k_router_dw<A><<<dim3(s.E, a.dw_router ? (s.H + 64 * A::VEC - 1) / (64 * A::VEC) : 1), 256, 0, st>>>(
        a, s.H, s.T * s.top_k, s.top_k);
  return hipGetLastError();
}

hipError_t launch_router_bwd(const moe_shape& s, const TrainPlan&, const RouterBwd& a,
                             hipStream_t st) {
  return s.act == MOE_DT_BF16 ? run<RowBf16>(s, a, st) : run<RowF32>(s, a, st);
}

}  // namespace moe
