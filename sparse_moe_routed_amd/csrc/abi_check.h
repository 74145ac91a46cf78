// Host-side checks shared by the C-ABI layers (moe_abi.cpp, block_abi.cpp).
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <initializer_list>

#include "moe_internal.h"

namespace moe {

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline size_t act_bytes(const moe_shape& s) { return s.act == MOE_DT_F32 ? 4 : 2; }

struct Span {
  const void* p;
  size_t n;
};

inline bool overlap(Span a, Span b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.n && b0 < a0 + a.n;
}

// Every output must be disjoint from every other output and every input.
inline bool any_alias(const Span* outs, int no, const Span* ins, int ni) {
  for (int i = 0; i < no; ++i) {
    for (int j = i + 1; j < no; ++j)
      if (overlap(outs[i], outs[j])) return true;
    for (int j = 0; j < ni; ++j)
      if (overlap(outs[i], ins[j])) return true;
  }
  return false;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int check_ptrs(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!p) return MOE_E_NULL;
  for (const void* p : ps)
    if (!aligned16(p)) return MOE_E_ALIGN;
  return MOE_OK;
}

inline int check_opt_ptr(const void* p) { return (p && !aligned16(p)) ? MOE_E_ALIGN : MOE_OK; }

inline int device_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_E_DEVICE; }

}  // namespace moe
