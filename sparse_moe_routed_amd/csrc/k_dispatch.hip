// Token rows in expert order and the gradients of dispatch, combine and the
// route weights (formulas: include/moe.h).  Bound by memory: every row is
// read and written once, in 16-byte chunks, and the T tokens are the unit of
// work, so that a token's own row is read once for its k slots.
// Measured, 4096 x 2560 bf16 top-10 (GPU time): dispatch 44.3 us (5.2 TB/s of
// 231 MB), weighted dispatch gradient 50.8 us (5.0 TB/s of 252 MB), combine
// gradient 91.2 us (4.8 TB/s of 441 MB), route gradient 5.5 us (latency).
#include <algorithm>

#include "moe_internal.h"
#include "row_device.h"

namespace moe {

// One wave per 64 chunks of a token's row: the chunk stays in registers while
// it is stored to each of the k rows.
template <class A, bool WEIGHTED>
__global__ __launch_bounds__(256) void k_dispatch(const void* x, const int32_t* pair_row,
                                                  const float* w, void* rows, int T, int H, int k,
                                                  int P) {
  constexpr int V = A::VEC;
  const int parts = (H / V + 63) / 64;
  const int unit = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const int t = unit / parts, c = unit - t * parts;
  if (t >= T) return;
  const int lane = threadIdx.x & 63;
  typedef RowRef<A, false, false> Row;
  const u32x4_t v = Row(x, static_cast<size_t>(t) * H, H).load(c, 64, lane);
  const int32_t* pr = pair_row + static_cast<size_t>(t) * k;
  for (int j0 = 0; j0 < k; j0 += 64) {
    const Slots<WEIGHTED> slots(pr, w + static_cast<size_t>(t) * k, j0, k, P);
    const int n = min(k - j0, 64);
    for (int u = 0; u < n; ++u) {
      const int r = slots.row(u);
      if (r < 0) continue;
      const Row row(rows, static_cast<size_t>(r) * H, H);
      if constexpr (WEIGHTED) {
        float f[V];
        A::unpack(v, f);
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] *= slots.weight(u);
        row.store(c, 64, lane, f);
      } else {
        row.store_raw(c, 64, lane, v);
      }
    }
  }
}

// Slots whose rows are requested together: with top_k up to 16 a chunk's
// sum is one round of loads.
constexpr int kSlotBatch = 16;

// dots[j * waves + wave]: a wave's share of slot j's dot product, over the
// chunks of the row that it has seen (LDS; lane 0 of the wave keeps it).
__device__ __forceinline__ void add_dot(float* dots, int j, float v, bool first) {
  v = wave_sum_f32(v);
  if ((threadIdx.x & 63) == 0) {
    float* d = dots + j * (blockDim.x >> 6) + (threadIdx.x >> 6);
    *d = first ? v : *d + v;
  }
}

// dw[j]: the waves' shares in wave order.
__device__ __forceinline__ void store_dots(const float* dots, float* dw, int k) {
  const int waves = blockDim.x >> 6;
  __syncthreads();
  for (int j = threadIdx.x; j < k; j += blockDim.x) {
    float s = dots[j * waves];
    for (int i = 1; i < waves; ++i) s += dots[j * waves + i];
    dw[j] = s;
  }
}

// A workgroup per token: the sum over its slots' rows and, with DW, each
// row's dot product with x.
template <class A, bool WEIGHTED, bool DW, bool STREAM>
__global__ __launch_bounds__(1024) void k_dispatch_bwd(const void* drows, const int32_t* pair_row,
                                                       const float* w, const void* x,
                                                       const void* dx_in, void* dx, float* dw,
                                                       int H, int k, int P) {
  typedef RowRef<A, false, STREAM> Row;
  constexpr int V = A::VEC;
  constexpr u32x4_t zero = {0u, 0u, 0u, 0u};
  extern __shared__ float dots[];
  const int nt = blockDim.x, tid = threadIdx.x;
  const size_t t = blockIdx.x;
  for (int i = 0; i * nt * V < H; ++i) {
    u32x4_t xr, ar;
    if constexpr (DW) xr = Row(x, t * H, H).load_once(i, nt, tid);
    ar = dx_in ? Row(dx_in, t * H, H).load_once(i, nt, tid) : zero;
    float acc[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
    for (int j0 = 0; j0 < k; j0 += kSlotBatch) {
      u32x4_t v[kSlotBatch];
      const Slots<WEIGHTED> slots(pair_row + t * k, w + t * k, j0, k, P);
#pragma unroll
      for (int q = 0; q < kSlotBatch; q += 4)
        if (j0 + q < k)
#pragma unroll
          for (int u = q; u < q + 4; ++u) v[u] = Row::slot(drows, slots.row(u), H).load_once(i, nt, tid);
#pragma unroll
      for (int u = 0; u < kSlotBatch; ++u) {
        float dot = 0.f;
        if (slots.row(u) >= 0) {
          const float wj = slots.weight(u);
          float f[V], xv[V];
          A::unpack(v[u], f);
          if constexpr (DW) A::unpack(xr, xv);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            acc[e] = fmaf(wj, f[e], acc[e]);
            if constexpr (DW) dot = fmaf(f[e], xv[e], dot);
          }
        }
        if constexpr (DW)
          if (j0 + u < k) add_dot(dots, j0 + u, dot, i == 0);
      }
    }
    float a[V];
    A::unpack(ar, a);
#pragma unroll
    for (int e = 0; e < V; ++e) a[e] += acc[e];
    Row(dx, t * H, H).store(i, nt, tid, a);
  }
  if constexpr (DW) store_dots(dots, dw + t * k, k);
}

// A workgroup per token: its gradient row times the weight to each slot's
// row and, with DW, the slots' dot products with it.
template <class A, bool DW, bool STREAM>
__global__ __launch_bounds__(1024) void k_combine_bwd(const void* dout, const void* y,
                                                      const int32_t* pair_row, const float* w,
                                                      void* dy, float* dw, int H, int k, int P) {
  typedef RowRef<A, false, STREAM> Row;
  constexpr int V = A::VEC;
  extern __shared__ float dots[];
  const int nt = blockDim.x, tid = threadIdx.x;
  const size_t t = blockIdx.x;
  for (int i = 0; i * nt * V < H; ++i) {
    const u32x4_t gr = Row(dout, t * H, H).load_once(i, nt, tid);
    for (int j0 = 0; j0 < k; j0 += kSlotBatch) {
      u32x4_t v[kSlotBatch];
      const Slots<true> slots(pair_row + t * k, w + t * k, j0, k, P);
      if constexpr (DW)
#pragma unroll
        for (int q = 0; q < kSlotBatch; q += 4)
          if (j0 + q < k)
#pragma unroll
            for (int u = q; u < q + 4; ++u) v[u] = Row::slot(y, slots.row(u), H).load_once(i, nt, tid);
#pragma unroll
      for (int u = 0; u < kSlotBatch; ++u) {
        float dot = 0.f;
        const int r = slots.row(u);
        if (r >= 0) {
          const float wj = slots.weight(u);
          float g[V], f[V];
          A::unpack(gr, g);
          if constexpr (DW) {
            A::unpack(v[u], f);
#pragma unroll
            for (int e = 0; e < V; ++e) dot = fmaf(g[e], f[e], dot);
          }
#pragma unroll
          for (int e = 0; e < V; ++e) g[e] *= wj;
          Row(dy, static_cast<size_t>(r) * H, H).store(i, nt, tid, g);
        }
        if constexpr (DW)
          if (j0 + u < k) add_dot(dots, j0 + u, dot, i == 0);
      }
    }
  }
  if constexpr (DW) store_dots(dots, dw + t * k, k);
}

// Orders this wave's LDS accesses (they execute in program order; no other
// wave shares the data, so no barrier).
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A wave per token puts its row of dlogits together in LDS.
__global__ __launch_bounds__(256) void k_route_bwd(const int32_t* __restrict__ ids,
                                                   const float* __restrict__ w,
                                                   const float* __restrict__ dw,
                                                   float* __restrict__ dlogits, int T, int E,
                                                   int k) {
  extern __shared__ f32x4_t route_rows[];   // [4][pitch / 4]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, pitch = (E + 3) / 4 * 4;
  const size_t t = static_cast<size_t>(blockIdx.x) * 4 + wave;
  if (t >= static_cast<size_t>(T)) return;
  // the first 64 slots in registers, requested together
  int id = -1;
  float wj = 0.f, dj = 0.f;
  if (lane < k) {
    id = ids[t * k + lane];
    wj = w[t * k + lane];
    dj = dw[t * k + lane];
  }
  f32x4_t* row4 = route_rows + wave * (pitch / 4);
  float* row = reinterpret_cast<float*>(row4);
  for (int e = lane; e < pitch / 4; e += 64) row4[e] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  float s = wj * dj;
  for (int j = lane + 64; j < k; j += 64) s = fmaf(w[t * k + j], dw[t * k + j], s);
  s = wave_sum_f32(s);
  wave_lds_fence();
  if (id >= 0 && id < E) row[id] = wj * (dj - s);
  for (int j = lane + 64; j < k; j += 64) {
    const int e = ids[t * k + j];
    if (e >= 0 && e < E) row[e] = w[t * k + j] * (dw[t * k + j] - s);
  }
  wave_lds_fence();
  float* out = dlogits + t * E;
  if (E % 4 == 0) {
    for (int e = lane; e < E / 4; e += 64) *reinterpret_cast<f32x4_t*>(out + 4 * e) = row4[e];
  } else {
    for (int e = lane; e < E; e += 64) out[e] = row[e];
  }
}

hipError_t launch_dispatch(const moe_shape& s, const void* x, const int32_t* pair_row,
                           const float* w, void* rows, hipStream_t st) {
  const bool bf = s.act == MOE_DT_BF16;
  const int parts = (s.H / (bf ? 8 : 4) + 63) / 64;
  const unsigned blocks = (static_cast<unsigned>(s.T) * parts + 3) / 4;
  auto kern = bf ? (w ? k_dispatch<RowBf16, true> : k_dispatch<RowBf16, false>)
                 : (w ? k_dispatch<RowF32, true> : k_dispatch<RowF32, false>);
  hipLaunchKernelGGL(kern, dim3(blocks), dim3(256), 0, st, x, pair_row, w, rows, s.T, s.H, s.top_k,
                     s.T * s.top_k);
  return hipGetLastError();
}

// Threads of a token's workgroup: one chunk each, up to `most`; a longer row
// takes rounds of as many.
static int token_threads(const moe_shape& s, int most) {
  const int chunks = s.H / (s.act == MOE_DT_BF16 ? 8 : 4), rounds = (chunks + most - 1) / most;
  return ((chunks + rounds - 1) / rounds + 63) / 64 * 64;
}

// The dispatch gradient with dw holds the slots' rows until the dots are
// summed, and one workgroup past 512 threads fills a CU.  Once there are more
// tokens than CUs, two smaller ones hide each other's waits (top-8 bf16, up
// to 1024 threads against 512: 512 x 7168 16.7 / 14.4 us, 1024 x 5120
// 23.9 / 20.1, 2048 x 7168 65.0 / 58.1; 256 x 7168 9.5 / 10.4).  The combine
// gradient and the plain sum gain nothing (2048 x 5504 83.8 / 88.8 and
// 38.7 / 42.2).
static int dispatch_bwd_threads(const moe_shape& s, const float* dw) {
  return token_threads(s, dw && s.T > 256 ? 512 : 1024);
}

// LDS of the dot products (at most 1024 slots x 16 waves x 4 bytes = 64 KB).
static size_t dot_bytes(const moe_shape& s, int nt, const float* dw) {
  return dw ? static_cast<size_t>(s.top_k) * (nt / 64) * sizeof(float) : 0;
}

template <class A, bool STREAM>
static auto dispatch_bwd_kernel(bool weighted, bool dw) {
  return dw         ? k_dispatch_bwd<A, true, true, STREAM>
         : weighted ? k_dispatch_bwd<A, true, false, STREAM>
                    : k_dispatch_bwd<A, false, false, STREAM>;
}

template <class A, bool STREAM>
static auto combine_bwd_kernel(bool dw) {
  return dw ? k_combine_bwd<A, true, STREAM> : k_combine_bwd<A, false, STREAM>;
}

static bool streams_rows(const moe_shape& s) {
  return streams_slots(static_cast<size_t>(s.T) * s.top_k * s.H * (s.act == MOE_DT_BF16 ? 2 : 4));
}

hipError_t launch_dispatch_bwd(const moe_shape& s, const void* drows, const int32_t* pair_row,
                               const float* w, const void* x, const void* dx_in, void* dx,
                               float* dw, hipStream_t st) {
  const int nt = dispatch_bwd_threads(s, dw);
  const bool bf = s.act == MOE_DT_BF16, stream = streams_rows(s);
  auto kern = bf ? (stream ? dispatch_bwd_kernel<RowBf16, true>(w, dw)
                           : dispatch_bwd_kernel<RowBf16, false>(w, dw))
                 : (stream ? dispatch_bwd_kernel<RowF32, true>(w, dw)
                           : dispatch_bwd_kernel<RowF32, false>(w, dw));
  hipLaunchKernelGGL(kern, dim3(s.T), dim3(nt), dot_bytes(s, nt, dw), st, drows, pair_row, w, x,
                     dx_in, dx, dw, s.H, s.top_k, s.T * s.top_k);
  return hipGetLastError();
}

hipError_t launch_combine_bwd(const moe_shape& s, const void* dout, const void* y,
                              const int32_t* pair_row, const float* w, void* dy, float* dw,
                              hipStream_t st) {
  const int nt = token_threads(s, 1024);
  const bool bf = s.act == MOE_DT_BF16, stream = streams_rows(s);
  auto kern = bf ? (stream ? combine_bwd_kernel<RowBf16, true>(dw)
                           : combine_bwd_kernel<RowBf16, false>(dw))
                 : (stream ? combine_bwd_kernel<RowF32, true>(dw)
                           : combine_bwd_kernel<RowF32, false>(dw));
  hipLaunchKernelGGL(kern, dim3(s.T), dim3(nt), dot_bytes(s, nt, dw), st, dout, y, pair_row, w, dy,
                     dw, s.H, s.top_k, s.T * s.top_k);
  return hipGetLastError();
}

hipError_t launch_route_bwd(const moe_shape& s, const int32_t* ids, const float* w,
                            const float* dw, float* dlogits, hipStream_t st) {
  hipLaunchKernelGGL(k_route_bwd, dim3((s.T + 3) / 4), dim3(256),
                     4 * ((s.E + 3) / 4 * 4) * sizeof(float), st, ids, w, dw, dlogits, s.T, s.E,
                     s.top_k);
  return hipGetLastError();
}

}  // namespace moe
