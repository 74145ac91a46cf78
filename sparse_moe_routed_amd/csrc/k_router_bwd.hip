// Gradient of the router's product.
//
// Only the top_k selected logits of a token have a gradient, so both products
// are sparse: dx gathers top_k rows of w_router per token, dw_router sums the
// tokens of an expert's rows.  4 P H flops against 3 T H a + E H (a + 4) bytes:
// bound by memory and, through the gathers, by the caches (4096 tokens, 10 of 512
// experts, H 2560, bf16: two gathers of 210 MB, dx 18.8 us, dw_router 30.4).  dx alone, in
// calls in a row, gathers 12.5 TB/s at H 2048 (one pass of 256 threads), 2560 (a second
// pass with a quarter of them) and 4096 alike: other workgroups fill that pass.
#include "moe_internal.h"
#include "train_device.h"

namespace moe {

// Up to here every thread takes the dot product w . dw of a token's slots itself,
// where one launch makes all outputs and where two do: the order of the sum is the
// same, whatever outputs are asked for.
constexpr int kOwnDot = 16;

// w . dw of a token's slots
__device__ __forceinline__ float slots_dot(const RouterBwd& a, size_t p0, int k) {
  float dot = 0.f;
  for (int j = 0; j < k; ++j) dot = fmaf(a.w[p0 + j], a.dw[p0 + j], dot);
  return dot;
}

// One workgroup per token: dl of its pairs, then dx.  JOINT: dl is not kept.
template <class A, bool JOINT>
__device__ __forceinline__ void dx_token(const RouterBwd& a, int H, int E, int k, int block) {
  typedef typename A::T T;
  constexpr int V = A::VEC, DEEP = 4;
  __shared__ float dl[1024];
  __shared__ int expert[1024];
  __shared__ float part[4];
  const size_t p0 = static_cast<size_t>(block) * k;
  float dot = 0.f;
  if (JOINT || k <= kOwnDot) {
    dot = slots_dot(a, p0, k);
  } else {
    for (int j = threadIdx.x; j < k; j += 256) dot = fmaf(a.w[p0 + j], a.dw[p0 + j], dot);
    dot = wave_sum_f32(dot);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
    __syncthreads();
    dot = (part[0] + part[1]) + (part[2] + part[3]);
  }
  for (int j = threadIdx.x; j < k; j += 256) {
    const float d = a.w[p0 + j] * (a.dw[p0 + j] - dot);
    const int e = a.ids[p0 + j];
    dl[j] = d;
    expert[j] = static_cast<uint32_t>(e) < static_cast<uint32_t>(E) ? e : -1;   // -1: a dropped pair
    if constexpr (!JOINT) a.dl[p0 + j] = d;
  }
  __syncthreads();
  if (!a.dx) return;
  const T* wr = static_cast<const T*>(a.w_router);
  const size_t row = static_cast<size_t>(block) * H;
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
template <class A>
__global__ __launch_bounds__(256) void k_router_dx(RouterBwd a, int H, int E, int k) {
  dx_token<A, false>(a, H, E, k, blockIdx.x);
}

// One workgroup per expert and LANES 16-byte columns; its lane groups share the
// rows.  Tokens and gradients of 64 WAVES rows are read at once, into LDS, and
// every lane has eight rows of x on their way.  Workgroups that run together
// work on the same columns, so that the rows of x stay in the caches: 4096
// tokens, 10 of 512 experts, H 2560, bf16 gather 210 MB in 29.8 us; columns of
// 1024 bytes take 44.8 and eight waves of 256 bytes 44.5.  Without the rows of
// eight loads together it was 112.
template <class A, int WAVES, int LANES, bool JOINT>
__device__ __forceinline__ void dw_columns(const RouterBwd& a, int H, int P, PairDiv slots, int e, int column) {
  typedef typename A::T T;
  constexpr int V = A::VEC, THREADS = 64 * WAVES, GROUPS = THREADS / LANES, DEEP = 8;
  __shared__ uint32_t token[THREADS];
  __shared__ float grad[THREADS];
  __shared__ float sums[GROUPS][LANES * V + 4];
  __shared__ float bias[WAVES];
  const int tid = threadIdx.x, g = tid / LANES;
  const int h = (column * LANES + tid % LANES) * V;
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
      const uint32_t t = slots.div(p);
      float d;
      if constexpr (JOINT)
        d = a.w[p] * (a.dw[p] - slots_dot(a, static_cast<size_t>(t) * slots.k, slots.k));
      else
        d = a.dl[p];
      token[tid] = t;
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
      const int c = column * LANES * V + i;
      float sum = sums[0][i];
#pragma unroll
      for (int j = 1; j < GROUPS; ++j) sum += sums[j][i];
      if (c < H) a.dw_router[static_cast<size_t>(e) * H + c] = sum;
    }
  if (a.dbias && column == 0 && tid == 0) {
    db = bias[0];
#pragma unroll
    for (int j = 1; j < WAVES; ++j) db += bias[j];
    a.dbias[e] = db;
  }
}
template <class A, int WAVES, int LANES>
__global__ __launch_bounds__(64 * WAVES) void k_router_dw(RouterBwd a, int H, int P, PairDiv slots) {
  dw_columns<A, WAVES, LANES, false>(a, H, P, slots, blockIdx.x, blockIdx.y);
}

// Both in one launch, with the experts' workgroups first.
template <class A, int LANES>
__global__ __launch_bounds__(256) void k_router(RouterBwd a, int H, int E, int P, PairDiv slots, int columns) {
  const int block = blockIdx.x;
  if (block < E * columns)
    dw_columns<A, 4, LANES, true>(a, H, P, slots, block % E, block / E);
  else
    dx_token<A, true>(a, H, E, slots.k, block - E * columns);
}

template <class A, int WAVES, int LANES>
static hipError_t run_dw(const moe_shape& s, const RouterBwd& a, hipStream_t st) {
  constexpr int COLS = LANES * A::VEC;
  k_router_dw<A, WAVES, LANES><<<dim3(s.E, a.dw_router ? (s.H + COLS - 1) / COLS : 1), 64 * WAVES, 0, st>>>(
      a, s.H, s.T * s.top_k, PairDiv::of(s.top_k));
  return hipGetLastError();
}

template <class A, int LANES>
static hipError_t run_joint(const moe_shape& s, const RouterBwd& a, hipStream_t st) {
  const int columns = a.dw_router ? (s.H + LANES * A::VEC - 1) / (LANES * A::VEC) : 1;
  k_router<A, LANES><<<s.E * columns + (a.dx ? s.T : 0), 256, 0, st>>>(a, s.H, s.E, s.T * s.top_k,
                                                                      PairDiv::of(s.top_k), columns);
  return hipGetLastError();
}

template <class A>
static hipError_t run(const moe_shape& s, const RouterBwd& a, hipStream_t st) {
  // Few workgroups: narrower columns and more waves for the experts' many rows.
  const bool few = static_cast<long long>(s.E) * s.H < 512 * 32 * A::VEC;
  // A small call is its launches (333 tokens top-3 of 60, 384 float32: 8.4 -> 4.8 us;
  // 1500 top-4 of 128, 1280 float32, 31 MB of gathered rows: 13.1 -> 9.9); at 41 MB the
  // dot products taken again cost as much, at 210 MB a third more.
  const long long P = static_cast<long long>(s.T) * s.top_k;
  if (P > 0 && s.top_k <= kOwnDot && (a.dw_router || a.dbias) && P <= 512ll * s.E &&
      P * s.H * static_cast<int>(sizeof(typename A::T)) <= 32 << 20)
    return few ? run_joint<A, 16>(s, a, st) : run_joint<A, 32>(s, a, st);
  if (s.T > 0) {
    k_router_dx<A><<<s.T, 256, 0, st>>>(a, s.H, s.E, s.top_k);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  if (!a.dw_router && !a.dbias) return hipSuccess;
  return few ? run_dw<A, 16, 16>(s, a, st) : run_dw<A, 4, 32>(s, a, st);
}

hipError_t launch_router_bwd(const moe_shape& s, const RouterBwd& a, hipStream_t st) {
  return s.act == MOE_DT_BF16 ? run<RowBf16>(s, a, st) : run<RowF32>(s, a, st);
}

}  // namespace moe
