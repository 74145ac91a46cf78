// 8-bit checkpoints of activations, written and read back.
//
// 32 consecutive elements share a scale 2^e; a thread holds 8 of them (float32
// or bf16, 16 or 32 bytes in), four threads find the group's largest magnitude
// by two exchanges within the wave.  Bound by memory: a + 33/32 bytes per
// element each way (a = 2 or 4): 32768 x 2560 bf16 is written in 43 us (5.9 TB/s;
// median of 12 runs 50) and read back in 37 (6.8).
#include "moe_internal.h"
#include "train_device.h"

namespace moe {

template <class E>
__global__ __launch_bounds__(256) void k_save8(const typename E::T* __restrict__ v, size_t n8,
                                               uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const size_t step = static_cast<size_t>(gridDim.x) * 256;
  // n8 is a multiple of 4, so the four threads of a group go together
  for (size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; i < n8; i += step) {
    float a[8];
    load_vals<E>(v + i * 8, a);
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(a[j]) & 0x7fffffffu);
    top = max(top, dpp_u32<kDppXor1>(top));
    top = max(top, dpp_u32<kDppXor2>(top));
    const uint32_t b = scale8(top);
    const float inv = inverse8(b);
    *reinterpret_cast<u32x2_t*>(codes + i * 8) = u32x2_t{codes8(a, inv), codes8(a + 4, inv)};
    if ((i & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(b);
  }
}

template <class E>
__global__ __launch_bounds__(256) void k_restore8(const uint8_t* __restrict__ codes,
                                                  const uint8_t* __restrict__ scales, size_t n8,
                                                  typename E::T* __restrict__ v) {
  const size_t step = static_cast<size_t>(gridDim.x) * 256;
  for (size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; i < n8; i += step) {
    const u32x2_t c = *reinterpret_cast<const u32x2_t*>(codes + i * 8);
    const float f = factor8(scales[i >> 2]);
    float a[8];
    values8(c[0], f, a);
    values8(c[1], f, a + 4);
    store_vals<E>(v + i * 8, a);
  }
}

static int grid8(size_t n8) {
  const size_t g = (n8 + 255) / 256;
  return static_cast<int>(g < 8192 ? g : 8192);
}

hipError_t launch_save8(bool f32, size_t n, const void* v, int8_t* codes, uint8_t* scales,
                        hipStream_t st) {
  uint8_t* c = reinterpret_cast<uint8_t*>(codes);
  if (f32)
    k_save8<TF32><<<grid8(n / 8), 256, 0, st>>>(static_cast<const float*>(v), n / 8, c, scales);
  else
    k_save8<TBf16><<<grid8(n / 8), 256, 0, st>>>(static_cast<const uint16_t*>(v), n / 8, c, scales);
  return hipGetLastError();
}

hipError_t launch_restore8(bool f32, size_t n, const int8_t* codes, const uint8_t* scales, void* v,
                           hipStream_t st) {
  const uint8_t* c = reinterpret_cast<const uint8_t*>(codes);
  if (f32)
    k_restore8<TF32><<<grid8(n / 8), 256, 0, st>>>(c, scales, n / 8, static_cast<float*>(v));
  else
    k_restore8<TBf16><<<grid8(n / 8), 256, 0, st>>>(c, scales, n / 8, static_cast<uint16_t*>(v));
  return hipGetLastError();
}

}  // namespace moe
