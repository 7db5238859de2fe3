// Root-mean-square norm with the residual's addition: what its entry points and kernels share.
#pragma once
#include "common.h"
#include "gmem.h"

namespace ftmoe {

struct NormForward {
  const void *x, *residual, *weight;  // residual: null for 0
  void *sum, *y;                      // null: not wanted, as the following
  int8_t* codes;
  float* scale;
  int64_t ld_x, ld_residual, ld_sum, ld_y, ld_codes;
  int32_t rows, cols;
  double eps;
};

struct NormBackward {
  const void *sum, *weight, *dy, *dsum;  // dsum: null for 0
  void *dx, *dresidual;                  // null: not wanted
  void* dweight;                         // one group of rows writes it itself, null: not so
  float* part;                           // [groups][norm_part_ld]: sums of dy s r over each group's rows, null: not wanted
  float* stats;                          // rows that no workgroup holds: a NormSlope of each
  int64_t ld_sum, ld_y, ld_residual, ld_x;
  int32_t rows, cols, groups;
  double eps;
};

// floats between two groups' parts: whole 16-byte pieces
#ifdef __HIPCC__
__host__ __device__
#endif
inline int64_t norm_part_ld(int32_t cols) { return (int64_t(cols) + 3) / 4 * 4; }
// groups of rows whose weight gradients are summed apart
int norm_groups(int32_t rows, int32_t cols);
// Rows that one workgroup takes one after the other, with the weight's gradient,
// in one launch instead of two: bf16, 2048 / 7168 columns, us, one launch of
// 1 / 2 / 3 rows 3.3 / 4.2 / 5.2 and 4.7 / 6.7 / 8.6, two launches 5.6 and 7.2.
constexpr int kNormOnce = 2;

// norm_rows.hip: rows that a workgroup's registers hold; norm_any.hip: all others
bool norm_rows(int32_t cols);
hipError_t launch_norm_rows(int dtype, int residual_dtype, const NormForward& a, hipStream_t s);
hipError_t launch_norm_rows(int dtype, int residual_dtype, const NormBackward& a, hipStream_t s);

hipError_t launch_norm(int dtype, int residual_dtype, const NormForward& a, hipStream_t s);
hipError_t launch_norm_backward(int dtype, int residual_dtype, const NormBackward& a, hipStream_t s);
// dweight = the sum of the groups' parts, in order
hipError_t launch_norm_join(int dtype, const float* part, int32_t groups, int32_t cols, void* dweight, hipStream_t s);

}  // namespace ftmoe
