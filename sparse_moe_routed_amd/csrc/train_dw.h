// Arguments of the weight gradients' kernels.
#pragma once

#include "moe_internal.h"
#include "train_rows.h"

namespace moe {

struct DwArgs {
  const void *dg, *du, *h, *dy, *x;
  void *dgate, *dup, *ddown;
  const int32_t *offsets, *sorted_pair;
  float* part;   // float32 partial sums [parts][3][E][I H] (parts > 1)
  PairDiv slots;
  int E, H, I, P;
  int parts;   // of an expert's rows; 0: tiles of 256 x 256
  int mean_stages;   // of an expert's rows (256 x 256)
  int strip;   // neighbouring tiles of a workgroup
  int unit;    // neighbouring strips on one XCD
};

// The rows' gradient by the same launch, tiles of 32 rows (parts 1 only).
struct DxArgs {
  RowArgs rows;
  const void *gate, *up;
  void* drows;
  int blocks;   // workgroups, a multiple of 8
};

hipError_t launch_dw(const moe_shape& s, const DwArgs& a, const DxArgs* x, hipStream_t st);

}  // namespace moe
