// Token rows in expert order and the gradients of dispatch, combine and the
// route weights (formulas: include/moe.h).
//
// One workgroup per token, element by element.
#include "moe_internal.h"
#include "row_device.h"

namespace moe {

template <class A>
__global__ __launch_bounds__(256) void k_dispatch(const typename A::T* x, const int32_t* pair_row,
                                                  const float* w, typename A::T* rows, int H,
                                                  int k, int P) {
  const size_t t = blockIdx.x;
  for (int j = 0; j < k; ++j) {
    const int r = pair_row[t * k + j];
    if (r < 0 || r >= P) continue;
    for (int h = threadIdx.x; h < H; h += 256) {
      const typename A::T v = x[t * H + h];
      rows[static_cast<size_t>(r) * H + h] = w ? A::put(w[t * k + j] * A::get(v)) : v;
    }
  }
}

template <class A>
__global__ __launch_bounds__(256) void k_dispatch_bwd(const typename A::T* drows,
                                                      const int32_t* pair_row, const float* w,
                                                      const typename A::T* x,
                                                      const typename A::T* dx_in,
                                                      typename A::T* dx, float* dw, int H, int k,
                                                      int P) {
  __shared__ float red[2][4];
  const size_t t = blockIdx.x;
  for (int h = threadIdx.x; h < H; h += 256) {
    float s = 0.f;
    for (int j = 0; j < k; ++j) {
      const int r = pair_row[t * k + j];
      if (r < 0 || r >= P) continue;
      s = fmaf(w ? w[t * k + j] : 1.f, A::get(drows[static_cast<size_t>(r) * H + h]), s);
    }
    if (dx_in) s += A::get(dx_in[t * H + h]);
    dx[t * H + h] = A::put(s);
  }
  if (!dw) return;
  for (int j = 0; j < k; ++j) {
    const int r = pair_row[t * k + j];
    float s = 0.f;
    if (r >= 0 && r < P)
      for (int h = threadIdx.x; h < H; h += 256)
        s = fmaf(A::get(x[t * H + h]), A::get(drows[static_cast<size_t>(r) * H + h]), s);
    s = row_sum<false>(s, red[j & 1]);
    if (threadIdx.x == 0) dw[t * k + j] = s;
  }
}

template <class A>
__global__ __launch_bounds__(256) void k_combine_bwd(const typename A::T* dout,
                                                     const typename A::T* y,
                                                     const int32_t* pair_row, const float* w,
                                                     typename A::T* dy, float* dw, int H, int k,
                                                     int P) {
  __shared__ float red[2][4];
  const size_t t = blockIdx.x;
  for (int j = 0; j < k; ++j) {
    const int r = pair_row[t * k + j];
    const float wj = w[t * k + j];
    float s = 0.f;
    if (r >= 0 && r < P)
      for (int h = threadIdx.x; h < H; h += 256) {
        const float d = A::get(dout[t * H + h]);
        const size_t i = static_cast<size_t>(r) * H + h;
        dy[i] = A::put(wj * d);
        if (dw) s = fmaf(d, A::get(y[i]), s);
      }
    if (!dw) continue;
    s = row_sum<false>(s, red[j & 1]);
    if (threadIdx.x == 0) dw[t * k + j] = s;
  }
}

// One wave per token; the row of dlogits is put together in LDS.
__global__ __launch_bounds__(64) void k_route_bwd(const int32_t* ids, const float* w,
                                                  const float* dw, float* dlogits, int E, int k) {
  __shared__ float row[1024];
  const size_t t = blockIdx.x;
  float s = 0.f;
  for (int j = threadIdx.x; j < k; j += 64) s = fmaf(w[t * k + j], dw[t * k + j], s);
  s = wave_sum_f32(s);
  for (int e = threadIdx.x; e < E; e += 64) row[e] = 0.f;
  __syncthreads();
  for (int j = threadIdx.x; j < k; j += 64) {
    const int e = ids[t * k + j];
    if (e >= 0 && e < E) row[e] = w[t * k + j] * (dw[t * k + j] - s);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 64) dlogits[t * E + e] = row[e];
}

template <class A>
static hipError_t dispatch_t(const moe_shape& s, const void* x, const int32_t* pair_row,
                             const float* w, void* rows, hipStream_t st) {
  typedef typename A::T E;
  hipLaunchKernelGGL(k_dispatch<A>, dim3(s.T), dim3(256), 0, st, static_cast<const E*>(x), pair_row,
                     w, static_cast<E*>(rows), s.H, s.top_k, s.T * s.top_k);
  return hipGetLastError();
}

hipError_t launch_dispatch(const moe_shape& s, const void* x, const int32_t* pair_row,
                           const float* w, void* rows, hipStream_t st) {
  return s.act == MOE_DT_BF16 ? dispatch_t<RowBf16>(s, x, pair_row, w, rows, st)
                              : dispatch_t<RowF32>(s, x, pair_row, w, rows, st);
}

template <class A>
static hipError_t dispatch_bwd_t(const moe_shape& s, const void* drows, const int32_t* pair_row,
                                 const float* w, const void* x, const void* dx_in, void* dx,
                                 float* dw, hipStream_t st) {
  typedef typename A::T E;
  hipLaunchKernelGGL(k_dispatch_bwd<A>, dim3(s.T), dim3(256), 0, st, static_cast<const E*>(drows),
                     pair_row, w, static_cast<const E*>(x), static_cast<const E*>(dx_in),
                     static_cast<E*>(dx), dw, s.H, s.top_k, s.T * s.top_k);
  return hipGetLastError();
}

hipError_t launch_dispatch_bwd(const moe_shape& s, const void* drows, const int32_t* pair_row,
                               const float* w, const void* x, const void* dx_in, void* dx,
                               float* dw, hipStream_t st) {
  return s.act == MOE_DT_BF16
             ? dispatch_bwd_t<RowBf16>(s, drows, pair_row, w, x, dx_in, dx, dw, st)
             : dispatch_bwd_t<RowF32>(s, drows, pair_row, w, x, dx_in, dx, dw, st);
}

template <class A>
static hipError_t combine_bwd_t(const moe_shape& s, const void* dout, const void* y,
                                const int32_t* pair_row, const float* w, void* dy, float* dw,
                                hipStream_t st) {
  typedef typename A::T E;
  hipLaunchKernelGGL(k_combine_bwd<A>, dim3(s.T), dim3(256), 0, st, static_cast<const E*>(dout),
                     static_cast<const E*>(y), pair_row, w, static_cast<E*>(dy), dw, s.H, s.top_k,
                     s.T * s.top_k);
  return hipGetLastError();
}

hipError_t launch_combine_bwd(const moe_shape& s, const void* dout, const void* y,
                              const int32_t* pair_row, const float* w, void* dy, float* dw,
                              hipStream_t st) {
  return s.act == MOE_DT_BF16 ? combine_bwd_t<RowBf16>(s, dout, y, pair_row, w, dy, dw, st)
                              : combine_bwd_t<RowF32>(s, dout, y, pair_row, w, dy, dw, st);
}

hipError_t launch_route_bwd(const moe_shape& s, const int32_t* ids, const float* w,
                            const float* dw, float* dlogits, hipStream_t st) {
  hipLaunchKernelGGL(k_route_bwd, dim3(s.T), dim3(64), 0, st, ids, w, dw, dlogits, s.E, s.top_k);
  return hipGetLastError();
}

}  // namespace moe
