// A router's balance: what the entry points and kernels share.
#pragma once
#include "common.h"
#include "gmem.h"

namespace ftmoe {

struct BalanceForward {
  const void* logits;
  const uint8_t* valid;  // null: all
  int32_t* sel;
  float* w;
  int32_t* counts;  // [E + 1]
  float* loss;
  // by workgroup: sums of p and choices [groups][ld_part], tokens counted [groups]
  float* part_p;
  int32_t *part_c, *part_v;
  double* share;     // of the loss, without its factor: of 16 experts each
  int32_t* arrived;  // workgroups that have written theirs
  int64_t ld;
  int32_t tokens, experts, top_k, groups, ld_part;
  float weight;
};

struct BalanceBackward {
  const void* logits;
  const uint8_t* valid;
  const int32_t* sel;
  const float* w;
  const int32_t* counts;
  const float *dw, *dloss;  // null: none; 1
  void* dlogits;
  int64_t ld;
  int32_t tokens, experts, top_k;
  float weight;
};

int balance_groups(int32_t tokens);
// experts' places in a part: whole lanes of a wave
inline int balance_width(int32_t experts) { return experts <= 64 ? 64 : experts <= 128 ? 128 : experts <= 256 ? 256 : 512; }
hipError_t launch_balance(int dtype, const BalanceForward& a, hipStream_t s);
hipError_t launch_balance_backward(int dtype, const BalanceBackward& a, hipStream_t s);

}  // namespace ftmoe
