// The norms around a block, forward: the norm before it, and combine, norm,
// gate, residual scale and next norm after it in one pass (formulas:
// include/moe.h).
//
// Bound by memory (a few flop per byte): every input is read once into
// registers, every output written once, float32 in between; the sum of
// squares of the next norm is taken while the output is formed.  Few rows are
// bound by latency: all loads are issued before the first sum (not those of
// bf16 rows of odd length, whose chunks wait one by one: RowRef<A, true>).
// Measured (GPU time): norm_in 1 x 2560 bf16 1.9 us; norm_out with a full
// sigmoid gate and the next norm, 4096 x 2560 bf16, 20.4 us (5.1 TB/s of 105
// MB); combine, norm and next norm, 512 x 2560 top-10, 8.8 us (3.9 TB/s of 34
// MB: two workgroups per CU, one round), 4096 x 2560 top-10 52.3 us a call (5.2
// TB/s of 273 MB), float32 107.8.
#include <algorithm>

#include "moe_internal.h"
#include "row_device.h"

namespace moe {

struct FwdArgs {
  NormFwd a;
  moe_norm n;
  int P;
};

// Thread `tid` of the `nt` threads of a row holds chunks tid, tid + nt, ...
// (C of them).  L: how threads share rows (RowShare); only a workgroup's row
// needs barriers.  An absent matrix is held as zeros (weights: offset 1), so
// that nothing but loads depends on it.
template <class A, int L, int C, bool COMBINE, int EDGE, bool STREAM, int GATE>
__global__ __launch_bounds__(L ? 256 : 1024) void k_norm_fwd(FwdArgs p) {
  typedef RowRef<A, EDGE == kEdgeOdd, STREAM> Row;
  typedef RowShare<L> Share;
  constexpr bool WAVE = Share::WAVE;
  constexpr int V = A::VEC;
  __shared__ float red[WAVE ? 1 : 2][16];
  const int nt = Share::threads(), tid = Share::place();
  const int t0 = WAVE ? __builtin_amdgcn_readfirstlane(
                            (blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6)) * Share::ROWS)
                      : blockIdx.x;
  if (WAVE && t0 >= p.n.T) return;
  const int t = t0 + Share::lane_row(), H = p.n.H;
  const uint32_t flags = p.n.flags;
  const bool normed = !(flags & MOE_N_NO_NORM);
  auto load = [&](const void* m, int i) { return Row(m, 0, H).load(i, nt, tid); };
  auto load_once = [&](const void* m, int i) {
    return row_ref<A, L, EDGE, STREAM>(m, t, p.n.T, H).load_once(i, nt, tid);
  };
  auto store = [&](void* m, int i, const float(&x)[V]) {
    row_ref<A, L, EDGE, STREAM>(m, t, p.n.T, H).store(i, nt, tid, x);
  };

  // everything is requested before the first use where registers allow
  constexpr bool EARLY = WAVE || C <= 2;
  constexpr u32x4_t zero = {0u, 0u, 0u, 0u};
  auto weight = [&](int i) { return normed ? load(p.a.w, i) : zero; };
  auto gate = [&](int i) { return load_once(p.a.gate, i); };
  auto residual = [&](int i) { return p.a.residual ? load_once(p.a.residual, i) : zero; };
  u32x4_t wr[EARLY ? C : 1], gr[EARLY ? C : 1], rr[EARLY ? C : 1], nr[EARLY ? C : 1];
  if constexpr (EARLY) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      wr[i] = weight(i);
      if constexpr (GATE != kGateRow) gr[i] = gate(i);
      rr[i] = residual(i);
      if (p.a.n_next) nr[i] = load(p.a.w_next, i);
    }
  }
  float v[C][V];
  if constexpr (COMBINE) {
    // slots in batches: the batch's rows are all requested, then added, j ascending
    constexpr int KB = C == 1 ? 16 : C == 2 ? 4 : C == 4 ? 2 : 1;
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] = 0.f;
    const int32_t* pr = p.a.pair_row + static_cast<size_t>(t) * p.a.k;
    const float* tw = p.a.topk_w + static_cast<size_t>(t) * p.a.k;
    for (int j0 = 0; j0 < p.a.k; j0 += KB) {
      u32x4_t y[KB][C];
      const Slots<true> slots(pr, tw, j0, p.a.k, p.P);
      constexpr int G = KB < 4 ? KB : 4;   // slots past the last one go in groups
#pragma unroll
      for (int q = 0; q < KB; q += G)
        if (j0 + q < p.a.k)
#pragma unroll
          for (int u = q; u < q + G; ++u)
#pragma unroll
            for (int i = 0; i < C; ++i) y[u][i] = Row::slot(p.a.y, slots.row(u), H).load_once(i, nt, tid);
#pragma unroll
      for (int q = 0; q < KB; q += G)
        if (j0 + q < p.a.k)
#pragma unroll
          for (int u = q; u < q + G; ++u) {
            const float w = slots.weight(u);
#pragma unroll
            for (int i = 0; i < C; ++i) {
              float f[V];
              A::unpack(y[u][i], f);
#pragma unroll
              for (int e = 0; e < V; ++e) v[i][e] = fmaf(w, f[e], v[i][e]);
            }
          }
    }
    if (p.a.z_out)
#pragma unroll
      for (int i = 0; i < C; ++i) store(p.a.z_out, i, v[i]);
  } else {
    u32x4_t zr[C];
#pragma unroll
    for (int i = 0; i < C; ++i) zr[i] = load_once(p.a.z, i);
#pragma unroll
    for (int i = 0; i < C; ++i) A::unpack(zr[i], v[i]);
  }
  float gt = 1.f;
  if (flags & MOE_N_GATE_TOKEN) {
    const float* g = static_cast<const float*>(p.a.gate);
    gt = Share::PACK ? (t < p.n.T ? g[t] : 0.f) : uniform_load(g + t0);
    if (flags & MOE_N_GATE_SIGMOID) gt = sigmoid<true>(gt);
  }
  float rs = 1.f;
  if (normed) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) ss = fmaf(v[i][e], v[i][e], ss);
    rs = rsqrtf(row_sum<L>(ss, red[0]) / H + p.n.eps);
  }
  const float offset = normed ? p.n.weight_offset : 1.f, factor = gt * p.n.branch_scale;
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    if constexpr (!EARLY) asm volatile("" ::: "memory");   // keep the loads of a chunk together
    float w[V], g[V], r[V];
    A::unpack(EARLY ? wr[i] : weight(i), w);
    A::unpack(EARLY ? rr[i] : residual(i), r);
    if constexpr (GATE != kGateRow) A::unpack(EARLY ? gr[i] : gate(i), g);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      v[i][e] = v[i][e] * rs * (w[e] + offset) * factor;
      if constexpr (GATE == kGateFull) v[i][e] *= g[e];
      if constexpr (GATE == kGateFullSigmoid) v[i][e] *= sigmoid<A::VEC == 4>(g[e]);
      v[i][e] = fmaf(p.n.residual_scale, r[e], v[i][e]);
      ss = fmaf(v[i][e], v[i][e], ss);   // zeros past the row's end
    }
    store(p.a.out, i, v[i]);
  }
  if (!p.a.n_next) return;
  const float rn = rsqrtf(row_sum<L>(ss, red[WAVE ? 0 : 1]) / H + p.n.eps);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    float f[V];
    A::unpack(EARLY ? nr[i] : load(p.a.w_next, i), f);
#pragma unroll
    for (int e = 0; e < V; ++e) v[i][e] *= rn * (f[e] + p.n.weight_offset);
    store(p.a.n_next, i, v[i]);
  }
}

typedef void (*FwdKernel)(FwdArgs);

template <class A, int EDGE, bool STREAM, int GATE>
static FwdKernel fwd_pack(int lanes) {
  switch (lanes) {
    case 8: return k_norm_fwd<A, 8, 1, false, EDGE, STREAM, GATE>;
    case 16: return k_norm_fwd<A, 16, 1, false, EDGE, STREAM, GATE>;
    default: return k_norm_fwd<A, 32, 1, false, EDGE, STREAM, GATE>;
  }
}

template <int EDGE, bool STREAM, int GATE>
static FwdKernel fwd_wave(int C) {
  switch (C) {
    case 1: return k_norm_fwd<RowBf16, 64, 1, false, EDGE, STREAM, GATE>;
    case 2: return k_norm_fwd<RowBf16, 64, 2, false, EDGE, STREAM, GATE>;
    case 3: return k_norm_fwd<RowBf16, 64, 3, false, EDGE, STREAM, GATE>;
    default: return k_norm_fwd<RowBf16, 64, 5, false, EDGE, STREAM, GATE>;
  }
}

template <class A, bool COMBINE, int EDGE, bool STREAM, int GATE>
static FwdKernel fwd_block(int C) {
  switch (C) {
    case 1: return k_norm_fwd<A, 0, 1, COMBINE, EDGE, STREAM, GATE>;
    case 2: return k_norm_fwd<A, 0, 2, COMBINE, EDGE, STREAM, GATE>;
    case 4: return k_norm_fwd<A, 0, 4, COMBINE, EDGE, STREAM, GATE>;
    case 8: return k_norm_fwd<A, 0, 8, COMBINE, EDGE, STREAM, GATE>;
    default:   // float32: 16
      return k_norm_fwd<A, 0, 64 / A::VEC, COMBINE, EDGE, STREAM, GATE>;
  }
}

template <class A, bool COMBINE, int GATE>
static hipError_t fwd(const FwdArgs& p, hipStream_t st) {
  // bf16 rows of odd length have kernels of their own (H % 128 == 0 with COMBINE)
  constexpr int ODD = A::VEC == 8 && !COMBINE ? kEdgeOdd : kEdgeWords;
  const int T = p.n.T, H = p.n.H, chunks = (H + A::VEC - 1) / A::VEC;
  const bool odd = ODD == kEdgeOdd && H % 2 != 0;
  const size_t row = H * sizeof(typename A::T);
  const bool stream = COMBINE ? streams_slots(p.P * row) : streams_matrix(T * row);
  // A wave per row saves the barriers and is the faster one while there are
  // rows to fill the card with single waves and a row is at most 5 chunks per
  // lane; few rows finish sooner with a thread per chunk.  norm_out with a
  // full gate, 2560 bf16: 1 row 4.4 us (wave) against 3.3 (workgroup), 512
  // rows 6.0 / 5.8, 2048 rows 12.7 / 13.8, 32768 rows 117 / 126.  float32
  // rows have twice the chunks: the workgroup is never slower there (4096 x
  // 1024: 19.1 / 16.2 us).  Rows of at most 32 chunks share a wave.
  const int many = T >= 1024;
  if (!COMBINE && many && chunks <= 32) {
    const int lanes = norm_pack_lanes(chunks), rows = 4 * 64 / lanes;
    auto kern = odd               ? fwd_pack<A, ODD, false, GATE>(lanes)
                : H % A::VEC != 0 ? fwd_pack<A, kEdgeCut, false, GATE>(lanes)
                : stream          ? fwd_pack<A, kEdgeWords, true, GATE>(lanes)
                                  : fwd_pack<A, kEdgeWords, false, GATE>(lanes);
    hipLaunchKernelGGL(kern, dim3((T + rows - 1) / rows), dim3(256), 0, st, p);
    return hipGetLastError();
  }
  if constexpr (!COMBINE && A::VEC == 8) {
    if (many && chunks <= 5 * 64) {
      const int C = (chunks + 63) / 64;
      auto kern = odd      ? fwd_wave<ODD, false, GATE>(C)
                  : stream ? fwd_wave<kEdgeWords, true, GATE>(C)
                           : fwd_wave<kEdgeWords, false, GATE>(C);
      hipLaunchKernelGGL(kern, dim3((T + 3) / 4), dim3(256), 0, st, p);
      return hipGetLastError();
    }
  }
  int C = 1;
  while (chunks > 1024 * C) C *= 2;
  const int nt = ((chunks + C - 1) / C + 63) / 64 * 64;
  auto kern = odd      ? fwd_block<A, COMBINE, ODD, false, GATE>(C)
              : stream ? fwd_block<A, COMBINE, kEdgeWords, true, GATE>(C)
                       : fwd_block<A, COMBINE, kEdgeWords, false, GATE>(C);
  hipLaunchKernelGGL(kern, dim3(T), dim3(nt), 0, st, p);
  return hipGetLastError();
}

template <class A, bool COMBINE>
static hipError_t fwd_gate(const FwdArgs& p, hipStream_t st) {
  if (!(p.n.flags & MOE_N_GATE_FULL)) return fwd<A, COMBINE, kGateRow>(p, st);
  return p.n.flags & MOE_N_GATE_SIGMOID ? fwd<A, COMBINE, kGateFullSigmoid>(p, st)
                                        : fwd<A, COMBINE, kGateFull>(p, st);
}

hipError_t launch_norm_fwd(const moe_norm& n, const NormFwd& a, hipStream_t st) {
  const FwdArgs p{a, n, n.T * a.k};
  if (n.act == MOE_DT_BF16) return a.y ? fwd_gate<RowBf16, true>(p, st) : fwd_gate<RowBf16, false>(p, st);
  return a.y ? fwd_gate<RowF32, true>(p, st) : fwd_gate<RowF32, false>(p, st);
}

}  // namespace moe
