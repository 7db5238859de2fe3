// Rows to 8-bit codes with one scale each: scale = fp32(max|x| / 127), code =
// x / scale rounded to the nearest integer, ties to even.
//
// The quotient is rounded correctly without a division: n = rint(x * r) with
// r about 1 / scale is within one of the result, and x - n * scale, which a
// fused multiply-add gives exactly (it is a multiple of the smaller unit in
// the last place of x and scale, and no larger than scale), says which
// neighbour is nearer and where a tie is.  So codes depend neither on the
// reciprocal's accuracy nor on the order in which a row is walked.
//
// Bound by HBM: each row is read once into registers and its codes are
// written once.
#include "dense.h"

namespace ftmoe {

namespace {

__device__ inline int row_code(float x, float s, float r) {
  float n = rintf(x * r);
  const float d = fmaf(-n, s, x), half = 0.5f * s;
  const bool odd = (int(n) & 1) != 0;
  if (d > half || (d == half && odd)) n += 1.0f;
  if (d < -half || (d == -half && odd)) n -= 1.0f;
  return int(fminf(fmaxf(n, -127.0f), 127.0f));
}

// 16 bytes of a row (4 or 8 neighbours) from column c; beyond the row's end, zeros.
template <typename E, int N>
__device__ __attribute__((always_inline)) inline void load16(const E* x, int c, int cols, float* v) {
  typedef E raw __attribute__((ext_vector_type(N)));
  typedef raw __attribute__((aligned(1))) any;
  const int cnt = cols - c;
  if (cnt >= N) {
    const raw e = gload<any>(x + c);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = float(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < cnt ? float(gload<E>(x + c + i)) : 0.f;
  }
}

// A row by THREADS threads, which keep up to GROUPS pieces of 16 bytes of it each;
// what a longer row has beyond that is read twice.
template <typename E, int THREADS, int GROUPS>
__global__ __launch_bounds__(THREADS) void k_int_quantize(const E* x, int64_t ld_x, int cols, int8_t* codes,
                                                          int64_t ld_codes, float* scale) {
  constexpr int N = 16 / int(sizeof(E)), kSweep = THREADS * N;
  const int64_t row = blockIdx.x;
  const E* xr = x + row * ld_x;
  int8_t* cr = codes + row * ld_codes;
  const int c0 = int(threadIdx.x) * N;
  // magnitudes compare as integers; infinities and NaN lie above every finite one
  uint32_t mx = 0;
  float v[GROUPS][N];
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) load16<E, N>(xr, c0 + g * kSweep, cols, v[g]);
  for (int c = c0 + GROUPS * kSweep; c < cols; c += kSweep) {
    float t[N];
    load16<E, N>(xr, c, cols, t);
#pragma unroll
    for (int i = 0; i < N; ++i) mx = max(mx, __float_as_uint(t[i]) & 0x7FFFFFFFu);
  }
#pragma unroll
  for (int g = 0; g < GROUPS; ++g)
#pragma unroll
    for (int i = 0; i < N; ++i) mx = max(mx, __float_as_uint(v[g][i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) mx = max(mx, uint32_t(__shfl_xor(int(mx), o)));
  if constexpr (THREADS > 64) {
    __shared__ uint32_t top[THREADS / 64];
    if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = mx;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) mx = max(mx, top[i]);
  }
  const bool finite = mx < 0x7F800000u;
  const float s = finite ? __uint_as_float(mx) / 127.0f : __uint_as_float(0x7FC00000u);
  if (threadIdx.x == 0) scale[row] = s;
  const bool live = finite && s > 0.f;
  // tiny scales are taken into the normal range, exactly, so that r is finite
  const float k = s < 0x1p-100f ? 0x1p100f : 1.0f;
  const float sk = live ? s * k : 1.0f, r = __builtin_amdgcn_rcpf(sk);
  auto put = [&](int c, const float* t) {
    typedef int8_t bytes __attribute__((ext_vector_type(N)));
    typedef bytes __attribute__((aligned(1))) any;
    bytes q;
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = int8_t(live ? row_code(t[i] * k, sk, r) : 0);
    if (c + N <= cols) {
      gstore<any>(cr + c, q);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (c + i < cols) gstore<int8_t>(cr + c + i, q[i]);
    }
  };
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) put(c0 + g * kSweep, v[g]);
  for (int c = c0 + GROUPS * kSweep; c < cols; c += kSweep) {
    float t[N];
    load16<E, N>(xr, c, cols, t);
    put(c, t);
  }
}

template <typename E>
hipError_t launch(int32_t rows, int32_t cols, const void* x, int64_t ld_x, int8_t* codes, int64_t ld_codes,
                  float* scale, hipStream_t s) {
  const E* e = static_cast<const E*>(x);
  // threads for which four pieces each hold the row, up to 256 x 4
  const int64_t bytes = int64_t(cols) * int64_t(sizeof(E));
  if (bytes <= 64 * 64)
    hipLaunchKernelGGL((k_int_quantize<E, 64, 4>), dim3(uint32_t(rows)), dim3(64), 0, s, e, ld_x, cols, codes, ld_codes,
                       scale);
  else
    hipLaunchKernelGGL((k_int_quantize<E, 256, 4>), dim3(uint32_t(rows)), dim3(256), 0, s, e, ld_x, cols, codes,
                       ld_codes, scale);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int_quantize(int dtype, int32_t rows, int32_t cols, const void* x, int64_t ld_x, int8_t* codes,
                               int64_t ld_codes, float* scale, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  if (dtype == FT_DT_F32) return launch<float>(rows, cols, x, ld_x, codes, ld_codes, scale, s);
  if (dtype == FT_DT_F16) return launch<_Float16>(rows, cols, x, ld_x, codes, ld_codes, scale, s);
  return launch<__bf16>(rows, cols, x, ld_x, codes, ld_codes, scale, s);
}

}  // namespace ftmoe
