// Gradient of the router's product.
//
// Only the top_k selected logits of a token have a gradient, so both products
// are sparse: dx gathers top_k rows of w_router per token, dw_router sums the
// tokens of an expert's rows.  4 P H flops against 3 T H a + E H (a + 4) bytes:
// bound by memory and, through the gathers, by the caches.
#include "moe_internal.h"
#include "train_device.h"

namespace moe {

// One workgroup per token: dl of its pairs, then dx.
template <class A>
__global__ __launch_bounds__(256) void k_router_dx(RouterBwd a, int H, int E, int k) {
  typedef typename A::T T;
  constexpr int V = A::VEC, DEEP = 4;
  __shared__ float dl[1024];
  __shared__ int expert[1024];
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
    const int e = a.ids[p0 + j];
    dl[j] = d;
    expert[j] = static_cast<uint32_t>(e) < static_cast<uint32_t>(E) ? e : -1;   // -1: a dropped pair
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
    for (int j = 0; j < k; j += DEEP) {
      u32x4_t q[DEEP];
#pragma unroll
      for (int i = 0; i < DEEP; ++i)
        q[i] = ld16(wr + static_cast<size_t>(max(expert[min(j + i, k - 1)], 0)) * H + h);
      sched_fence();
#pragma unroll
      for (int i = 0; i < DEEP; ++i) {
        if (j + i >= k || expert[j + i] < 0) continue;
        float r[V];
        A::unpack(q[i], r);
#pragma unroll
        for (int c = 0; c < V; ++c) v[c] = fmaf(dl[j + i], r[c], v[c]);
      }
    }
    *reinterpret_cast<u32x4_t*>(static_cast<T*>(a.dx) + row + h) = A::pack(v);
  }
}

// One workgroup per expert and LANES 16-byte columns; its lane groups share the
// rows.  Tokens and gradients of 64 WAVES rows are read at once, into LDS, and
// every lane has eight rows of x on their way.  Workgroups that run together
// work on the same columns, so that the rows of x stay in the caches: 4096
// tokens, 10 of 512 experts, H 2560, bf16 gather 210 MB in 29.8 us; columns of
// 1024 bytes take 44.8 and eight waves of 256 bytes 44.5.  Without the rows of
// eight loads together it was 112.
template <class A, int WAVES, int LANES>
__global__ __launch_bounds__(64 * WAVES) void k_router_dw(RouterBwd a, int H, int P, PairDiv slots) {
  typedef typename A::T T;
  constexpr int V = A::VEC, THREADS = 64 * WAVES, GROUPS = THREADS / LANES, DEEP = 8;
  __shared__ uint32_t token[THREADS];
  __shared__ float grad[THREADS];
  __shared__ float sums[GROUPS][LANES * V + 4];
  __shared__ float bias[WAVES];
  const int e = blockIdx.x, tid = threadIdx.x, g = tid / LANES;
  const int h = (blockIdx.y * LANES + tid % LANES) * V;
  const bool cols = a.dw_router && h < H;
  int row0 = 0, rows = 0;
  if (P > 0) {
    row0 = min(max(a.offsets[e], 0), P);
    rows = min(max(a.offsets[e + 1], row0), P) - row0;
  }
  const T* x = static_cast<const T*>(a.x) + h;
  float v[V] = {}, db = 0.f;
  for (int r0 = 0; r0 < rows; r0 += THREADS) {
    const int here = min(rows - r0, THREADS);
    if (tid < here) {
      const int p = min(max(a.sorted_pair[row0 + r0 + tid], 0), P - 1);
      const float d = a.dl[p];
      token[tid] = slots.div(p);
      grad[tid] = d;
      db += d;
    }
    __syncthreads();
    if (cols)
      for (int r = g; r < here; r += GROUPS * DEEP) {
        u32x4_t q[DEEP];
#pragma unroll
        for (int i = 0; i < DEEP; ++i)
          q[i] = ld16(x + static_cast<size_t>(token[min(r + i * GROUPS, here - 1)]) * H);
        sched_fence();
#pragma unroll
        for (int i = 0; i < DEEP; ++i) {
          const bool in = r + i * GROUPS < here;   // behind the last row: zeros
          const float d = in ? grad[r + i * GROUPS] : 0.f;
          float f[V];
          A::unpack(in ? q[i] : u32x4_t{0, 0, 0, 0}, f);
#pragma unroll
          for (int j = 0; j < V; ++j) v[j] = fmaf(d, f[j], v[j]);
        }
      }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < V; ++i) sums[g][tid % LANES * V + i] = v[i];
  db = wave_sum_f32(db);
  if ((tid & 63) == 0) bias[tid >> 6] = db;
  __syncthreads();
  if (a.dw_router)
    for (int i = tid; i < LANES * V; i += THREADS) {
      const int c = blockIdx.y * LANES * V + i;
      float sum = sums[0][i];
#pragma unroll
      for (int j = 1; j < GROUPS; ++j) sum += sums[j][i];
      if (c < H) a.dw_router[static_cast<size_t>(e) * H + c] = sum;
    }
  if (a.dbias && blockIdx.y == 0 && tid == 0) {
    db = bias[0];
#pragma unroll
    for (int j = 1; j < WAVES; ++j) db += bias[j];
    a.dbias[e] = db;
  }
}

template <class A, int WAVES, int LANES>
static hipError_t run_dw(const moe_shape& s, const RouterBwd& a, hipStream_t st) {
  constexpr int COLS = LANES * A::VEC;
  k_router_dw<A, WAVES, LANES><<<dim3(s.E, a.dw_router ? (s.H + COLS - 1) / COLS : 1), 64 * WAVES, 0, st>>>(
      a, s.H, s.T * s.top_k, PairDiv::of(s.top_k));
  return hipGetLastError();
}

template <class A>
static hipError_t run(const moe_shape& s, const RouterBwd& a, hipStream_t st) {
  if (s.T > 0) {
    k_router_dx<A><<<s.T, 256, 0, st>>>(a, s.H, s.E, s.top_k);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  if (!a.dw_router && !a.dbias) return hipSuccess;
  // Few workgroups: narrower columns and more waves for the experts' many rows.
  const bool few = static_cast<long long>(s.E) * s.H < 512 * 32 * A::VEC;
  return few ? run_dw<A, 16, 16>(s, a, st) : run_dw<A, 4, 32>(s, a, st);
}

hipError_t launch_router_bwd(const moe_shape& s, const RouterBwd& a, hipStream_t st) {
  return s.act == MOE_DT_BF16 ? run<RowBf16>(s, a, st) : run<RowF32>(s, a, st);
}

}  // namespace moe
