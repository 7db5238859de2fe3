// Root-mean-square norm: rows of any width, element by element.
//
// For rows that norm_rows.hip does not take (fewer than 8 columns, more than
// 16384).  Every row is read twice: for its sums, and for its values.  Here
// too: the join of the weight gradient's parts (512 x 7168: 4.9 us).
#include "norm_device.h"

namespace ftmoe {

namespace {

constexpr int kThreads = 256;

template <typename X, typename R>
__global__ __launch_bounds__(kThreads) void k_norm_any(NormForward a) {
  __shared__ double lds[3 * kThreads / 64];
  const int64_t row = int64_t(blockIdx.y) * kNormGrid + blockIdx.x;
  if (row >= a.rows) return;
  const X* x = static_cast<const X*>(a.x) + row * a.ld_x;
  const R* residual = a.residual ? static_cast<const R*>(a.residual) + row * a.ld_residual : nullptr;
  const X* weight = static_cast<const X*>(a.weight);
  R* sum = a.sum ? static_cast<R*>(a.sum) + row * a.ld_sum : nullptr;
  X* y = a.y ? static_cast<X*>(a.y) + row * a.ld_y : nullptr;
  int8_t* codes = a.codes ? a.codes + row * a.ld_codes : nullptr;
  auto at = [&](int c) { return double(float(gload<X>(x + c))) + (residual ? double(float(gload<R>(residual + c))) : 0.0); };

  NormSums t;
  for (int c = threadIdx.x; c < a.cols; c += kThreads) t.add(at(c), double(float(gload<X>(weight + c))));
  t.join<kThreads>(lds);
  const NormRow r(t, a.cols, a.eps);
  if (codes && threadIdx.x == 0) a.scale[row] = r.scale;
  for (int c = threadIdx.x; c < a.cols; c += kThreads) {
    const double s = at(c), sw = s * double(float(gload<X>(weight + c)));
    if (sum) gstore<R>(sum + c, R(float(s)));
    if (y) gstore<X>(y + c, X(float(sw * r.r)));
    if (codes) gstore<int8_t>(codes + c, int8_t(r.code(sw)));
  }
}

typedef float NormStats __attribute__((ext_vector_type(4)));  // a row's NormSlope, in one load

template <typename X, typename R, bool FAR>
__global__ __launch_bounds__(kThreads) void k_norm_stats_any(NormBackward a) {
  __shared__ double lds[2 * kThreads / 64];
  const int64_t row = int64_t(blockIdx.y) * kNormGrid + blockIdx.x;
  if (row >= a.rows) return;
  const R* sum = static_cast<const R*>(a.sum) + row * a.ld_sum;
  const X* dy = static_cast<const X*>(a.dy) + row * a.ld_y;
  const X* weight = static_cast<const X*>(a.weight);
  NormDots t;
  for (int c = threadIdx.x; c < a.cols; c += kThreads)
    t.add(float(gload<R>(sum + c)), float(gload<X>(dy + c)) * float(gload<X>(weight + c)));
  t.join<kThreads>(lds);
  const NormSlope<FAR> k(t, a.cols, a.eps);
  if (threadIdx.x == 0) {
    const NormStats v{k.r, k.m, k.up, 0.f};
    gstore<NormStats>(a.stats + 4 * row, v);
  }
}

// a column for each thread, the rows of a group one after the other
template <typename X, typename R, bool FAR>
__global__ __launch_bounds__(kThreads) void k_norm_grad_any(NormBackward a) {
  const int c = int(blockIdx.x) * kThreads + int(threadIdx.x);
  if (c >= a.cols) return;
  const float w = float(gload<X>(static_cast<const X*>(a.weight) + c));
  float dw = 0.f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float s = float(gload<R>(static_cast<const R*>(a.sum) + row * a.ld_sum + c));
    const float dy = float(gload<X>(static_cast<const X*>(a.dy) + row * a.ld_y + c));
    const NormStats v = gload<NormStats>(a.stats + 4 * row);
    const NormSlope<FAR> k(v[0], v[1], v[2]);
    const float n = k.n(s);
    float ds = k.ds(dy * w, n);
    if (a.dsum) ds += float(gload<R>(static_cast<const R*>(a.dsum) + row * a.ld_residual + c));
    if (a.dx) gstore<X>(static_cast<X*>(a.dx) + row * a.ld_x + c, X(ds));
    if (a.dresidual) gstore<R>(static_cast<R*>(a.dresidual) + row * a.ld_residual + c, R(ds));
    dw = fmaf(dy, n, dw);
  }
  if (a.part) a.part[int64_t(blockIdx.y) * norm_part_ld(a.cols) + c] = dw;
}

// 32 columns a workgroup: eight lanes have four each, 128 groups of lanes every 128th part.
constexpr int kJoin = 1024;
template <typename X>
__global__ __launch_bounds__(kJoin) void k_norm_join(const float* part, int groups, int cols, X* dweight) {
  typedef float floatx4 __attribute__((ext_vector_type(4)));
  __shared__ floatx4 lds[kJoin / 64][8];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t ld = norm_part_ld(cols);
  const int c0 = 32 * int(blockIdx.x), c = c0 + 4 * (tid & 7);
  floatx4 t{};
  if (c < cols) {
#pragma unroll 4
    for (int g = tid >> 3; g < groups; g += kJoin / 8) t += gload<floatx4>(part + g * ld + c);
  }
#pragma unroll
  for (int o = 8; o < 64; o <<= 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] += __shfl_xor(t[i], o);
  }
  if (lane < 8) lds[wave][lane] = t;
  __syncthreads();
  if (tid < 32 && c0 + tid < cols) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kJoin / 64; ++w) v += lds[w][tid >> 2][tid & 3];
    gstore<X>(dweight + c0 + tid, X(v));
  }
}

template <typename X, typename R>
hipError_t launch(const NormForward& a, hipStream_t s) {
  hipLaunchKernelGGL((k_norm_any<X, R>), norm_grid(a.rows), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <typename X, typename R, bool FAR>
hipError_t launch_backward(const NormBackward& a, hipStream_t s) {
  hipLaunchKernelGGL((k_norm_stats_any<X, R, FAR>), norm_grid(a.rows), dim3(kThreads), 0, s, a);
  const uint32_t across = uint32_t((a.cols + kThreads - 1) / kThreads);
  hipLaunchKernelGGL((k_norm_grad_any<X, R, FAR>), dim3(across, uint32_t(a.groups)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}
template <typename X, typename R>
hipError_t launch(const NormBackward& a, hipStream_t s) {
  return a.eps > 0.0 ? launch_backward<X, R, false>(a, s) : launch_backward<X, R, true>(a, s);
}

template <typename A>
hipError_t launch_types(int dtype, int residual_dtype, const A& a, hipStream_t s) {
  const bool same = dtype == residual_dtype;
  if (dtype == FT_DT_F32) return launch<float, float>(a, s);
  if (dtype == FT_DT_F16) return same ? launch<_Float16, _Float16>(a, s) : launch<_Float16, float>(a, s);
  return same ? launch<__bf16, __bf16>(a, s) : launch<__bf16, float>(a, s);
}

}  // namespace

int norm_groups(int32_t rows, int32_t cols) {
  const int32_t most = norm_rows(cols) ? 512 : 64;
  return rows < most ? rows : most;
}

hipError_t launch_norm(int dtype, int residual_dtype, const NormForward& a, hipStream_t s) {
  return norm_rows(a.cols) ? launch_norm_rows(dtype, residual_dtype, a, s) : launch_types(dtype, residual_dtype, a, s);
}
hipError_t launch_norm_backward(int dtype, int residual_dtype, const NormBackward& a, hipStream_t s) {
  return norm_rows(a.cols) ? launch_norm_rows(dtype, residual_dtype, a, s) : launch_types(dtype, residual_dtype, a, s);
}

hipError_t launch_norm_join(int dtype, const float* part, int32_t groups, int32_t cols, void* dweight, hipStream_t s) {
  const dim3 grid(uint32_t((cols + 31) / 32));
  if (dtype == FT_DT_F32)
    hipLaunchKernelGGL((k_norm_join<float>), grid, dim3(kJoin), 0, s, part, groups, cols, static_cast<float*>(dweight));
  else if (dtype == FT_DT_F16)
    hipLaunchKernelGGL((k_norm_join<_Float16>), grid, dim3(kJoin), 0, s, part, groups, cols,
                       static_cast<_Float16*>(dweight));
  else
    hipLaunchKernelGGL((k_norm_join<__bf16>), grid, dim3(kJoin), 0, s, part, groups, cols, static_cast<__bf16*>(dweight));
  return hipGetLastError();
}

}  // namespace ftmoe
