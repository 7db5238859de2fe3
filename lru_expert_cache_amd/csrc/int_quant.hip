// Rows to 8-bit codes with one scale each.
//
// Bound by HBM: each row is read once into registers and its codes are
// written once.  8192 x 7168, called over and over: bf16 33 us (5.3 TB/s read and
// written; with every element looked at closely, one by one, 56), fp32 60 us (4.9).
#include "int_quant.h"

namespace ftmoe {

namespace {

// A row by THREADS threads, which keep up to GROUPS pieces of 16 bytes of it each;
// what a longer row has beyond that is read twice.
template <typename E, int THREADS, int GROUPS>
__global__ __launch_bounds__(THREADS) void k_int_quantize(const E* x, int64_t ld_x, int cols, int8_t* codes,
                                                          int64_t ld_codes, float* scale) {
  constexpr int N = RowPiece<E>::N, kSweep = THREADS * N;
  const int64_t row = blockIdx.x;
  const E* xr = x + row * ld_x;
  int8_t* cr = codes + row * ld_codes;
  const int c0 = int(threadIdx.x) * N;
  const bool last = cols % N != 0 && threadIdx.x == 0;  // has the piece that the row ends in
  RowPiece<E> v[GROUPS], end;
  RowMax<E> most;
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) v[g].load(xr, c0 + g * kSweep, cols);
  if (last) {
    end.load_last(xr, cols);
    most.add(end);
  }
  for (int c = c0 + GROUPS * kSweep; c < cols; c += kSweep) {
    RowPiece<E> t;
    t.load(xr, c, cols);
    most.add(t);
  }
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) most.add(v[g]);
  uint32_t mx = most.bits();
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) mx = max(mx, uint32_t(__shfl_xor(int(mx), o)));
  if constexpr (THREADS > 64) {
    __shared__ uint32_t top[THREADS / 64];
    if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = mx;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) mx = max(mx, top[i]);
  }
  const RowScale q(mx);
  if (threadIdx.x == 0) scale[row] = q.scale;
  auto put = [&](int c, const RowPiece<E>& t) {
    if (c + N > cols) return;
    typedef uint32_t words __attribute__((ext_vector_type(N / 4)));
    typedef words __attribute__((aligned(1))) any;
    uint32_t b[N / 4];
    q.codes(t, b);
    words w;
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = b[i];
    gstore<any>(cr + c, w);
  };
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) put(c0 + g * kSweep, v[g]);
  for (int c = c0 + GROUPS * kSweep; c < cols; c += kSweep) {
    RowPiece<E> t;
    t.load(xr, c, cols);
    put(c, t);
  }
  if (last) {
    uint32_t b[N / 4];
    q.codes(end, b);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < cols % N) gstore<int8_t>(cr + cols / N * N + i, int8_t(b[i / 4] >> (i % 4 * 8)));
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
