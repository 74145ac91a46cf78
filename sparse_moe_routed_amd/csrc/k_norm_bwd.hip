// Gradient of the norms around a block (formulas: include/moe.h).  One pass:
// rs(z) and mean(g zh) come from two sums over the row, sum z^2 and
// sum G d w z, taken together while the row is in registers; dz, the gate's
// gradient and the row's share of dw follow from registers.  dw adds up in
// float32 registers over the rows of a wave (or workgroup), then over the
// waves of a workgroup in LDS, and a second launch adds the workgroups' rows
// of partial sums: no atomics, the same bits every time.  A single row is its
// own dw (1 x 2560 bf16 5.8 -> 3.2 us on the GPU without the second launch).
//
// Bound by memory.  Measured (GPU time, then k_norm_dw): 32768 x 2560 bf16
// with the residual path's gradient 128 + 4.8 us (5.2 TB/s of 671 MB), 4096 x
// 2560 with a full sigmoid gate 25.4 + 4.8 us (4.1 TB/s of 105 MB).
#include <algorithm>

#include "moe_internal.h"
#include "row_device.h"

namespace moe {

struct BwdArgs {
  NormBwd a;
  moe_norm n;
};

// L: how threads share rows (RowShare).  KEEP: the row stays in registers
// between the sums and the results (otherwise it is read again, from the
// cache).  An absent matrix is held as zeros (weights: offset 1), so that
// nothing but loads depends on it.
template <class A, int L, int C, int EDGE, bool STREAM, int GATE>
__global__ __launch_bounds__(!L ? 1024 : C == 1 ? 512 : 256) void k_norm_bwd(BwdArgs p) {
  typedef RowRef<A, EDGE == kEdgeOdd, STREAM> Row;
  typedef RowShare<L> Share;
  constexpr bool WAVE = Share::WAVE;
  constexpr int V = A::VEC;
  constexpr bool KEEP = WAVE || C <= 2;
  __shared__ float2 red[2][WAVE ? 1 : 16];
  extern __shared__ float colsum[];   // WAVE: the workgroup's dw
  const int nt = Share::threads(), tid = Share::place();
  const int wave = WAVE ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  const int waves = WAVE ? blockDim.x >> 6 : 1;
  const int H = p.n.H;
  const uint32_t flags = p.n.flags;
  const bool normed = !(flags & MOE_N_NO_NORM), sig = flags & MOE_N_GATE_SIGMOID;
  constexpr bool full = GATE != kGateRow;
  const float bs = p.n.branch_scale;
  // kept rows are read once; the others come back for the second pass
  auto load = [&](const void* m, int t, int i) {
    const auto row = row_ref<A, L, EDGE, STREAM>(m, t, p.n.T, H);
    return KEEP ? row.load_once(i, nt, tid) : row.load(i, nt, tid);
  };
  float acc[C][V];
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) acc[i][e] = 0.f;
  constexpr u32x4_t zero = {0u, 0u, 0u, 0u};
  const float offset = normed ? p.n.weight_offset : 1.f;
  auto load_w = [&](int i) { return normed ? Row(p.a.w, 0, H).load(i, nt, tid) : zero; };
  // where neither a norm nor the gate's gradient wants z, its rows are taken
  // as of no features: they read as zeros, without touching memory
  const int Hz = normed || p.a.dgate ? H : 0;
  auto load_z = [&](int t, int i) {
    const auto row = row_ref<A, L, EDGE, STREAM>(p.a.z, t, p.n.T, Hz);
    return KEEP ? row.load_once(i, nt, tid) : row.load(i, nt, tid);
  };
  auto load_s = [&](int t, int i) { return p.a.dres ? load(p.a.dres, t, i) : zero; };
  u32x4_t wr[KEEP ? C : 1];
  if constexpr (KEEP)
#pragma unroll
    for (int i = 0; i < C; ++i) wr[i] = load_w(i);
  int parity = 0;
  const int step = gridDim.x * waves * Share::ROWS;
  for (int t0 = (blockIdx.x * waves + wave) * Share::ROWS; t0 < p.n.T; t0 += step, parity ^= 1) {
    const int t = t0 + Share::lane_row();
    u32x4_t zr[KEEP ? C : 1], dr[KEEP ? C : 1], gr[KEEP ? C : 1], sr[KEEP ? C : 1];
    if constexpr (KEEP)
#pragma unroll
      for (int i = 0; i < C; ++i) {
        zr[i] = load_z(t, i);
        dr[i] = load(p.a.dout, t, i);
        if constexpr (full) gr[i] = load(p.a.gate, t, i);
        sr[i] = load_s(t, i);
      }
    // a token gate, or its sigmoid's tail, until the sums are there
    float gt = 1.f;
    if (!full && (flags & MOE_N_GATE_TOKEN)) {
      const float* g = static_cast<const float*>(p.a.gate);
      gt = Share::PACK ? (t < p.n.T ? g[t] : 0.f) : uniform_load(g + t0);
      if (sig) gt = sigmoid_tail<true>(gt);
    }
    // the full gate's factors; of a sigmoid its tail, kept for the second use
    constexpr bool KEEP_G = KEEP && GATE == kGateFullSigmoid;
    float gk[KEEP_G ? C : 1][V];
    auto gate = [&](int i, float(&g)[V]) {
      if constexpr (full) A::unpack(KEEP ? gr[i] : load(p.a.gate, t, i), g);
      if constexpr (GATE == kGateFullSigmoid)
#pragma unroll
        for (int e = 0; e < V; ++e) g[e] = sigmoid_tail<V == 4>(g[e]);
    };
    auto factor = [](float g) { return GATE == kGateFullSigmoid ? tail_sigmoid(g) : g; };
    float ss = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      if constexpr (!KEEP) asm volatile("" ::: "memory");   // keep the loads of a chunk together
      float z[V], d[V], w[V], g[V];
      A::unpack(KEEP ? zr[i] : load_z(t, i), z);
      A::unpack(KEEP ? dr[i] : load(p.a.dout, t, i), d);
      A::unpack(KEEP ? wr[i] : load_w(i), w);
      gate(i, g);
      if constexpr (KEEP_G)
#pragma unroll
        for (int e = 0; e < V; ++e) gk[i][e] = g[e];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float dw = d[e] * (w[e] + offset);
        ss = fmaf(z[e], z[e], ss);
        s1 = fmaf(full ? factor(g[e]) * dw : dw, z[e], s1);
      }
    }
    // the row is unpacked again after the sums: twice the registers would be
    // live if its float32 values were kept
    if constexpr (KEEP)
#pragma unroll
      for (int i = 0; i < C; ++i) {
        asm volatile("" : "+v"(zr[i]), "+v"(dr[i]), "+v"(wr[i]));
        if constexpr (full && !KEEP_G) asm volatile("" : "+v"(gr[i]));
        if constexpr (KEEP_G)   // nor the factors beside their tails
#pragma unroll
          for (int e = 0; e < V; ++e) asm volatile("" : "+v"(gk[i][e]));
      }
    const float2 s = row_sum2<L>(ss, s1, red[parity]);
    const float rs = normed ? rsqrtf(s.x / H + p.n.eps) : 1.f;
    s1 = bs * (rs * s.y);                                  // sum_h db zh (w) G_full
    if (!full && (flags & MOE_N_GATE_TOKEN) && p.a.dgate && tid == 0 && t < p.n.T)
      static_cast<float*>(p.a.dgate)[t] = s1 * (sig ? tail_slope(gt) : 1.f);
    if (!full && sig) gt = tail_sigmoid(gt);
    const float c = normed ? gt * s1 / H : 0.f;            // mean(g zh)
    const float bg = bs * gt;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      if constexpr (!KEEP) asm volatile("" ::: "memory");
      float z[V], d[V], w[V], g[V], r[V];
      A::unpack(KEEP ? zr[i] : load_z(t, i), z);
      A::unpack(KEEP ? dr[i] : load(p.a.dout, t, i), d);
      A::unpack(KEEP ? wr[i] : load_w(i), w);
      if constexpr (KEEP_G) {
#pragma unroll
        for (int e = 0; e < V; ++e) g[e] = gk[i][e];
      } else {
        gate(i, g);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        z[e] *= rs;
        w[e] += offset;
      }
      if constexpr (full) {
        if (p.a.dgate) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            r[e] = bs * d[e] * z[e] * w[e];
            if constexpr (GATE == kGateFullSigmoid) r[e] *= tail_slope(g[e]);
          }
          row_ref<A, L, EDGE, STREAM>(p.a.dgate, t, p.n.T, H).store(i, nt, tid, r);
        }
      }
      float sv[V];
      A::unpack(KEEP ? sr[i] : load_s(t, i), sv);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        d[e] *= full ? bg * factor(g[e]) : bg;
        acc[i][e] = fmaf(d[e], z[e], acc[i][e]);
        r[e] = d[e] * w[e];
        if (normed) r[e] = rs * fmaf(-z[e], c, r[e]);   // without a norm z may be infinite
        r[e] = fmaf(p.n.residual_scale, sv[e], r[e]);
      }
      row_ref<A, L, EDGE, STREAM>(p.a.dz, t, p.n.T, H).store(i, nt, tid, r);
    }
  }
  if (!p.a.dw) return;
  // the rows that share a wave
  if constexpr (Share::PACK)
#pragma unroll
    for (int m = L; m < 64; m *= 2)
#pragma unroll
      for (int e = 0; e < V; ++e) acc[0][e] += wave_shfl_xor(acc[0][e], m);
  // rows of `part` and colsum are norm_part_pitch(H) long: whole chunks
  const int pitch = norm_part_pitch(H);
  if (!WAVE && gridDim.x == 1) {   // nothing to add up
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int q = 0; q < V; q += 4) {
        const int h = (i * nt + tid) * V + q;
        if (h + 4 <= H) {
          *reinterpret_cast<f32x4_t*>(p.a.dw + h) = {acc[i][q], acc[i][q + 1], acc[i][q + 2], acc[i][q + 3]};
        } else {
#pragma unroll
          for (int e = 0; e < 3; ++e)
            if (h + e < H) p.a.dw[h + e] = acc[i][q + e];
        }
      }
    return;
  }
  float* part = p.a.part + static_cast<size_t>(blockIdx.x) * pitch;
  // WAVE: the waves add their sums in turn, the last one writes
  for (int k = 0; k < waves; ++k) {
    if (k == wave && (!Share::PACK || Share::lane_row() == 0))
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int q = 0; q < V; q += 4) {
          const int h = (i * nt + tid) * V + q;
          if (h < pitch) {
            f32x4_t v = {acc[i][q], acc[i][q + 1], acc[i][q + 2], acc[i][q + 3]};
            if (k > 0) v += *reinterpret_cast<f32x4_t*>(colsum + h);
            *reinterpret_cast<f32x4_t*>((k == waves - 1 ? part : colsum) + h) = v;
          }
        }
    if (k < waves - 1) __syncthreads();
  }
}

// dw[h] = sum over G rows of part: 32 columns per workgroup, each by 32
// threads that take the rows in turn (up to 16 requested together), then
// added in LDS in a fixed order.
__global__ __launch_bounds__(1024) void k_norm_dw(const float* __restrict__ part,
                                                  float* __restrict__ dw, int G, int H,
                                                  int pitch) {
  __shared__ float sum[32][33];
  const int col = threadIdx.x & 31, by = threadIdx.x >> 5;
  const int h = blockIdx.x * 32 + col;
  float s = 0.f;
  for (int g0 = by; g0 < G; g0 += 32 * 16) {
    float v[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      const int g = g0 + 32 * u;
      v[u] = g < G && h < H ? part[static_cast<size_t>(g) * pitch + h] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < 16; ++u) s += v[u];
  }
  sum[by][col] = s;
  __syncthreads();
  // thread (col, by) now holds row col of column by
  s = sum[col][by];
#pragma unroll
  for (int m = 16; m > 0; m /= 2) s += __shfl_xor(s, m, 32);
  if (col == 0 && blockIdx.x * 32 + by < static_cast<unsigned>(H)) dw[blockIdx.x * 32 + by] = s;
}

typedef void (*BwdKernel)(BwdArgs);

template <class A, int EDGE, bool STREAM, int GATE>
static BwdKernel bwd_pack(int lanes) {
  switch (lanes) {
    case 8: return k_norm_bwd<A, 8, 1, EDGE, STREAM, GATE>;
    case 16: return k_norm_bwd<A, 16, 1, EDGE, STREAM, GATE>;
    default: return k_norm_bwd<A, 32, 1, EDGE, STREAM, GATE>;
  }
}

template <class A, int EDGE, bool STREAM, int GATE>
static BwdKernel bwd_kernel(int lanes, int C) {
  if (lanes > 0 && lanes < 64) return bwd_pack<A, EDGE, STREAM, GATE>(lanes);
  if (lanes == 64) switch (C) {
      case 1: return k_norm_bwd<A, 64, 1, EDGE, STREAM, GATE>;
      case 2: return k_norm_bwd<A, 64, 2, EDGE, STREAM, GATE>;
      case 3: return k_norm_bwd<A, 64, 3, EDGE, STREAM, GATE>;
      default: return k_norm_bwd<A, 64, 5, EDGE, STREAM, GATE>;
    }
  switch (C) {
    case 1: return k_norm_bwd<A, 0, 1, EDGE, STREAM, GATE>;
    case 2: return k_norm_bwd<A, 0, 2, EDGE, STREAM, GATE>;
    case 4: return k_norm_bwd<A, 0, 4, EDGE, STREAM, GATE>;
    case 8: return k_norm_bwd<A, 0, 8, EDGE, STREAM, GATE>;
    default: return k_norm_bwd<A, 0, 64 / A::VEC, EDGE, STREAM, GATE>;   // float32: 16
  }
}

template <class A, int GATE>
static void bwd(const BwdArgs& p, int G, hipStream_t st) {
  const int H = p.n.H, chunks = (H + A::VEC - 1) / A::VEC;
  const int lanes = norm_bwd_lanes(p.n);
  int C = 1, nt = 64 * norm_bwd_waves(p.n);
  if (lanes) {
    C = (chunks + 63) / 64;
  } else {
    while (chunks > 1024 * C) C *= 2;
    nt = ((chunks + C - 1) / C + 63) / 64 * 64;
  }
  const bool stream = streams_matrix(p.n.T * (H * sizeof(typename A::T)));
  constexpr int ODD = A::VEC == 8 ? kEdgeOdd : kEdgeWords;
  const bool pack = lanes > 0 && lanes < 64;
  auto kern = A::VEC == 8 && H % 2      ? bwd_kernel<A, ODD, false, GATE>(lanes, C)
              : pack && H % A::VEC != 0 ? bwd_pack<A, kEdgeCut, false, GATE>(lanes)
              : stream                  ? bwd_kernel<A, kEdgeWords, true, GATE>(lanes, C)
                                        : bwd_kernel<A, kEdgeWords, false, GATE>(lanes, C);
  hipLaunchKernelGGL(kern, dim3(G), dim3(nt), lanes && p.a.dw ? norm_part_pitch(H) * sizeof(float) : 0, st, p);
}

template <class A>
static void bwd_gate(const BwdArgs& p, int G, hipStream_t st) {
  if (!(p.n.flags & MOE_N_GATE_FULL))
    bwd<A, kGateRow>(p, G, st);
  else if (p.n.flags & MOE_N_GATE_SIGMOID)
    bwd<A, kGateFullSigmoid>(p, G, st);
  else
    bwd<A, kGateFull>(p, G, st);
}

hipError_t launch_norm_bwd(const moe_norm& n, const NormBwd& a, hipStream_t st) {
  const int G = norm_bwd_groups(n);
  const BwdArgs p{a, n};
  if (n.T > 0) {
    if (n.act == MOE_DT_BF16)
      bwd_gate<RowBf16>(p, G, st);
    else
      bwd_gate<RowF32>(p, G, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.dw && (n.T == 0 || G > 1))
    hipLaunchKernelGGL(k_norm_dw, dim3((n.H + 31) / 32), dim3(1024), 0, st, a.part, a.dw, G, n.H,
                       norm_part_pitch(n.H));
  return hipGetLastError();
}

}  // namespace moe
