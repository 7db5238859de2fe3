// Low-rank adapters beside a projection: what the entry points and kernels share.
#pragma once
#include "common.h"
#include "gmem.h"

namespace ftmoe {

struct Adapters {
  const void* x;
  const int32_t* ids;
  const void *a, *b;
  const float* scale;  // null: 1
  const void* base;    // null: 0
  void* y;
  float* h;            // [T][R]: A x
  int64_t ld_x, ld_a, ld_b, ld_base, ld_y;
  int32_t tokens, in, out, rank, count;
  bool in_place;       // y is base
};

hipError_t launch_adapters(int dtype, int base_dtype, int out_dtype, const Adapters& a, hipStream_t s);

}  // namespace ftmoe
